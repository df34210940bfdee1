// Low-rank adapters of many requests beside one shared projection. Token t uses
// adapter a = ids[t] (none if outside [0, n)), with down matrix A_a [R, H], up
// matrix B_a [N, R] and scale s_a:
//   v_t = A_a x_t  (FP32),        out_t = bf16(base_t + s_a B_a v_t),
// and for the gradient dy of out
//   du_t = s_a B_a^T dy_t,        dx_t = bf16(base_t + A_a^T du_t),
//   dA_a = sum_t du_t x_t^T,      dB_a = s_a sum_t dy_t v_t^T.
// R is small (8 .. 128), so x, dy, base and the outputs are what has to move;
// the matrices of one adapter stay in the caches while its tokens pass.
//
// Grouping. Tokens need not be sorted, and no plan is kept between calls. The
// first kernel of a call takes 1024 tokens (a span) at a time, puts them into an
// order in which the tokens of an adapter are neighbours, and cuts that order into
// units of at most 64 tokens of one adapter, whose rows are gathered into blocks of
// 16 (the width of one MFMA). Every workgroup of the span does so for itself, in
// LDS; one of them leaves the order and the units in the workspace for the kernels
// that follow. Requests that are runs of tokens are taken as they stand; otherwise
// the span is sorted.
//
// Bits of a token do not depend on the other tokens of the call: a column of an
// MFMA depends on its own operand column only, and how a sum over H (or N) is
// cut into parts follows from H (or N) alone.
//
// All products run on v_mfma_f32_16x16x32_bf16 (lane l holds row or column
// l % 16 and the eight k of group l / 16; the result lane holds column l % 16
// and rows 4 (l / 16) + 0..3). FP32 factors (v, du) enter as sums of BF16
// values: two (16 significant bits) where the result is rounded to BF16 (8
// bits), three where it stays FP32, which holds all 24 bits of an FP32 value.
//
// The time of a call is that of its passes over the rows: two forward, four backward (reduction,
// expansion, gradients, and the sum of the gradients' shares). Small calls cost their launches.
#include "device.h"
#include "kernels.h"

namespace pmoe {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 64;    // tokens of one unit at most
constexpr int kSpan = 1024;  // tokens that are grouped together
constexpr int kNone = -1;  // adapter of a unit of tokens without one
// Boundaries up to which a span is not sorted. Sorting costs 1 us; units of single tokens cost
// more: n = 12 adapters over T = 128 tokens in mixed order take 15.8 us a call, unsorted 50.
constexpr int kMostRuns = 16;

__device__ __forceinline__ floatx4 mfma16(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Loads and stores at a 32-bit byte offset from a pointer that is the same in all lanes: the
// pointer stays in scalar registers. Offsets within a span of tokens or within one adapter's
// matrix, and within a window of 4096 tokens, are at most 2^27.
template <typename V>
__device__ __forceinline__ V load_at(const void* base, uint32_t offset) {
  return *reinterpret_cast<const V*>(static_cast<const char*>(base) + offset);
}
template <typename V>
__device__ __forceinline__ void store_at(void* base, uint32_t offset, V v) {
  *reinterpret_cast<V*>(static_cast<char*>(base) + offset) = v;
}
// A buffer that starts at such a pointer, and loads from it that are 0 where `on` is false:
// their offset lies behind the buffer's end, which the hardware's range check turns into zeros,
// so that a masked load needs neither a branch nor registers set beforehand. `scalar` is an
// offset that is the same in all lanes.
using Buffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buffer buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
template <typename V>
__device__ __forceinline__ V load_if(Buffer b, uint32_t offset, bool on, int scalar = 0) {
  const uint32_t o = on ? offset : 0x80000000u;
  if constexpr (sizeof(V) == 16)
    return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(b, o, scalar, 0));
  else if constexpr (sizeof(V) == 8)
    return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(b, o, scalar, 0));
  else if constexpr (sizeof(V) == 4)
    return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b32(b, o, scalar, 0));
  else
    return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b16(b, o, scalar, 0));
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 u) { return __builtin_bit_cast(bf16x8_t, u); }

__device__ __forceinline__ int adapter_of(const void* ids, int ids64, long t, int n) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[t] : static_cast<const int*>(ids)[t];
  return id >= 0 && id < n ? (int)id : -1;
}

// Waves of a reducing workgroup, and the longest part of a row that it takes. Above rank 32 a wave
// holds so many sums that a CU has room for twelve: three workgroups of four, of which one groups
// or adds up while the others load (with eight waves and parts of 2048: T = 1024, n = 4, H = 4096,
// R = 64 24.8 us a call, not 22.7). Up to rank 32 two of eight fit, and longer parts group each
// span less often (with four waves and parts of 1024: T = 8192, n = 6, H = 7168, R = 16 84.5 us, not 83.3).
__host__ __device__ constexpr int reduce_waves(int R) { return R <= 32 ? 8 : 4; }
__host__ __device__ constexpr int reduce_part(int R) { return 256 * reduce_waves(R); }

// Order and units of a span: unit u holds the places [start[u], start[u + 1]) of
// the order; key = adapter << 10 | token of the span, adapter n for none.
constexpr int kChunks = kSpan / 64;
struct SpanLds {
  uint32_t key[kSpan];
  uint16_t start[kSpan + 8];
  int table[16][kChunks];  // sort: keys of a digit in a chunk of 64, then the places before them
  int wave[2][8];
};
// The same in the workspace, one for each span: the order, and the units as
// {first place | tokens << 16, adapter}.
struct SpanOrder {
  uint32_t key[kSpan];
  uint2 unit[kSpan];
  int units;
  int pad[3];
};

// Inclusive sum and maximum over the lanes by data-parallel-primitive moves: 1, 2, 4 and 8
// lanes up within rows of 16, then the last lane of a row into the rows above.
template <int kCtrl, int kRows>
__device__ __forceinline__ int lane_move(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, kCtrl, kRows, 0xf, false);
}
__device__ __forceinline__ int wave_inclusive_sum(int v) {
  v += lane_move<0x111, 0xf>(0, v);
  v += lane_move<0x112, 0xf>(0, v);
  v += lane_move<0x114, 0xf>(0, v);
  v += lane_move<0x118, 0xf>(0, v);
  v += lane_move<0x142, 0xa>(0, v);
  v += lane_move<0x143, 0xc>(0, v);
  return v;
}
__device__ __forceinline__ int wave_inclusive_max(int v) {
  v = max(v, lane_move<0x111, 0xf>(v, v));
  v = max(v, lane_move<0x112, 0xf>(v, v));
  v = max(v, lane_move<0x114, 0xf>(v, v));
  v = max(v, lane_move<0x118, 0xf>(v, v));
  v = max(v, lane_move<0x142, 0xa>(v, v));
  v = max(v, lane_move<0x143, 0xc>(v, v));
  return v;
}

// Groups the tokens [t0, t0 + count) with a workgroup of kWaves; returns
// the number of units. Ends with a barrier.
template <int kWaves>
__device__ __forceinline__ int group_span(const void* ids, int ids64, long t0, int count, int n, SpanLds& l) {
  constexpr int kThreads = 64 * kWaves, kPer = kSpan / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid + kThreads * j;
    key[j] = 0xFFFFFFFFu;
    if (i < count) {
      const int a = adapter_of(ids, ids64, t0 + i, n);
      key[j] = (uint32_t)(a < 0 ? n : a) << 10 | (uint32_t)i;
    }
    l.key[i] = key[j];
  }
  __syncthreads();
  int edges = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid + kThreads * j;
    edges += __popcll(__ballot(i > 0 && i < count && key[j] >> 10 != l.key[max(i, 1) - 1] >> 10));
  }
  if (lane == 0) l.wave[0][wave] = edges;
  __syncthreads();
  edges = 0;
  for (int w = 0; w < kWaves; ++w) edges += l.wave[0][w];
  if (edges > kMostRuns) {
    // Stable sort by adapter, four bits at a time from the lowest: a key's place is the number of
    // keys with a smaller digit, plus those with its digit in the chunks before its own, plus
    // those among the lanes below (found by ballots on the digit's bits).
    const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
    for (int shift = 10; n >> (shift - 10) != 0; shift += 4) {
      for (int i = tid; i < 16 * kChunks; i += kThreads) (&l.table[0][0])[i] = 0;
      __syncthreads();
      int digit[kPer], rank[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool on = tid + kThreads * j < count;
        digit[j] = key[j] >> shift & 15;
        uint64_t match = __ballot(on);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint64_t set = __ballot(digit[j] >> b & 1);
          match &= digit[j] >> b & 1 ? set : ~set;
        }
        rank[j] = __popcll(match & below);
        if (on && rank[j] == 0) l.table[digit[j]][wave + kWaves * j] = __popcll(match);
      }
      __syncthreads();
      const int mine = tid < 16 * kChunks ? (&l.table[0][0])[tid] : 0;
      const int upto = wave_inclusive_sum(mine);
      if (lane == 63) l.wave[1][wave] = upto;
      __syncthreads();
      int before = upto - mine;
      for (int w = 0; w < wave; ++w) before += l.wave[1][w];
      if (tid < 16 * kChunks) (&l.table[0][0])[tid] = before;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (tid + kThreads * j < count)
          l.key[l.table[digit[j]][wave + kWaves * j] + rank[j]] = key[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] = l.key[tid + kThreads * j];
    }
  }
  // Units. Thread t looks at the places kPer t .. kPer t + kPer - 1.
  uint32_t before_key = tid > 0 ? l.key[kPer * tid - 1] : 0;
  int first[kPer], last = -1;  // the start of the group that a place belongs to, -1: further back
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t k = l.key[kPer * tid + j];
    if ((tid == 0 && j == 0) || k >> 10 != before_key >> 10) last = kPer * tid + j;
    first[j] = last;
    before_key = k;
  }
  const int upto = wave_inclusive_max(last);
  __syncthreads();  // every wave has read the edges
  if (lane == 63) l.wave[0][wave] = upto;
  int back = __shfl_up(upto, 1, 64);  // exclusive; lane 0 has none within the wave
  if (lane == 0) back = -1;
  __syncthreads();
  for (int w = 0; w < wave; ++w) back = max(back, l.wave[0][w]);
  int starts = 0;
  bool is[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int at = kPer * tid + j, from = first[j] >= 0 ? first[j] : back;
    is[j] = at < count && ((at - from) & (kUnit - 1)) == 0;
    starts += is[j];
  }
  int place = wave_inclusive_sum(starts);
  if (lane == 63) l.wave[1][wave] = place;
  place -= starts;
  __syncthreads();
  int units = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) place += l.wave[1][w];
    units += l.wave[1][w];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (is[j]) l.start[place++] = (uint16_t)(kPer * tid + j);
  if (tid == 0) l.start[units] = (uint16_t)count;
  __syncthreads();
  return units;
}

template <int kThreads>
__device__ __forceinline__ void keep_order(const SpanLds& l, int units, int count, int n, SpanOrder* o) {
  for (int i = threadIdx.x; i < count; i += kThreads) o->key[i] = l.key[i];
  for (int i = threadIdx.x; i < units; i += kThreads) {
    const uint32_t at = l.start[i], len = l.start[i + 1] - at;
    const int a = l.key[at] >> 10;
    o->unit[i] = make_uint2(at | len << 16, a == n ? kNone : a);
  }
  if (threadIdx.x == 0) o->units = units;
}

// ---------------------------------------------------------------- reduction over H (or N)
// A sum over a row of D elements is cut into parts of adapter_part_length(D, R) elements (a
// multiple of 64, at most reduce_part(R)), one workgroup each, whose waves take pieces of
// 64 elements in turn: together they read a row in long stretches.
static int adapter_parts(int D, int R) { return (D + reduce_part(R) - 1) / reduce_part(R); }
static int adapter_part_length(int D, int R) {
  const int parts = adapter_parts(D, R);
  return ((D + parts - 1) / parts + 63) / 64 * 64;
}

// Eight rows of kCols columns each, turned: op[b] gets the eight values of
// column b, ready as an MFMA operand. kCols is 1, 2, 4 or 8.
template <int kCols>
struct Rows8 {
  static constexpr int kWords = kCols < 2 ? 1 : kCols / 2;
  uint32_t w[8][kWords];
  __device__ __forceinline__ void load(int j, Buffer from, uint32_t offset, bool on, int scalar = 0) {
    if constexpr (kCols == 1) {
      w[j][0] = load_if<uint16_t>(from, offset, on, scalar);
    } else if constexpr (kCols == 2) {
      w[j][0] = load_if<uint32_t>(from, offset, on, scalar);
    } else if constexpr (kCols == 4) {
      const uint2 u = load_if<uint2>(from, offset, on, scalar);
      w[j][0] = u.x, w[j][1] = u.y;
    } else {
      const uint4 u = load_if<uint4>(from, offset, on, scalar);
      w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
    }
  }
  __device__ __forceinline__ bf16x8_t column(int b) const {
    const uint32_t sel = b & 1 ? 0x07060302u : 0x05040100u;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(w[2 * j + 1][b / 2], w[2 * j][b / 2], sel);
    return as_bf16x8(make_uint4(o[0], o[1], o[2], o[3]));
  }
};

// A block of 16 rows x 64 elements on its way to the MFMA operands. An operand wants lane
// (col, g) to hold eight elements of row col, which would make every lane of a load its own
// cache access. So eight neighbouring lanes load the 128 bytes of a row (16 bytes each), and
// the block is turned through 2 KB of LDS that belong to the wave alone (its LDS operations
// stay in order); chunk c of row r lies at chunk c ^ (r & 7), which keeps both sides free of
// bank conflicts.
struct Block16 {
  uint4 v[2];  // rows 8 j + lane / 8
  __device__ __forceinline__ void load(int j, Buffer from, uint32_t offset, bool on) {
    v[j] = load_if<uint4>(from, offset, on);
  }
  // lo: elements 8 g .. 8 g + 7 of row col, hi: 32 elements further
  __device__ __forceinline__ void turn(uint4* lds, int lane, bf16x8_t& lo, bf16x8_t& hi) const {
    const int row = lane >> 3, at = row * 8 + ((lane & 7) ^ row);
    lds[at] = v[0];
    lds[at + 64] = v[1];
    const int col = lane & 15, g = lane >> 4, swap = col & 7;
    lo = as_bf16x8(lds[col * 8 + (g ^ swap)]);
    hi = as_bf16x8(lds[col * 8 + ((g + 4) ^ swap)]);
  }
};

// part[y][place][r] = sum over the y-th part of in[t][k] * W_a[r][k] (kTrans: W_a[k][r]),
// t the token at the place of the order. blockIdx.y is a span and one of `share`
// workgroups that take its units (with R > 64 its half units) in turn.
// Operand row i of block b is r = NR i + b, so that a lane ends with 4 NR consecutive r of
// one token, and with kTrans a lane reads NR neighbouring columns of eight rows.
// Bound by the latency of grouping, loads and adding up, one after the other: T = 8192, n = 6,
// H = 7168, R = 16 takes 41 us where every token has an adapter, 117 MB at 2.9 TB/s. Loading the
// next 64 elements ahead gained 1% there and lost 6% with R = 32, for want of registers. Many
// adapters in mixed order read each matrix once a span: T = 8192, n = 64, R = 64 takes 230 us a
// call. A grid with the spans of one part side by side, not its parts, lost on the former (83 us a
// call -> 87).
template <int NR, bool kTrans>
__global__ __launch_bounds__(64 * reduce_waves(16 * NR), NR <= 2 ? 4 : NR <= 4 ? 3 : 2) void adapter_reduce_kernel(
    const uint16_t* __restrict__ in, const void* __restrict__ ids, int ids64, int T, int n, int D, int R,
    const uint16_t* __restrict__ W, int length, int share, SpanOrder* __restrict__ orders,
    float* __restrict__ part) {
  constexpr int kWaves = reduce_waves(16 * NR);
  constexpr int NF = NR <= 4 ? 4 : 2;      // row blocks of an item: a unit, or half a unit
  __shared__ __align__(16) SpanLds lds;
  __shared__ uint4 turn[kWaves][2][128];
  __shared__ floatx4 red[kWaves][NR][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4, row8 = lane >> 3, chunk = lane & 7;
  const int sp = blockIdx.y / share, mine = blockIdx.y % share;
  const long t0 = (long)sp * kSpan;
  const int count = (int)min((long)kSpan, T - t0);
  const int units = group_span<kWaves>(ids, ids64, t0, count, n, lds);
  if (mine == 0 && blockIdx.x == 0) keep_order<64 * kWaves>(lds, units, count, n, orders + sp);
  const int k_begin = blockIdx.x * length + wave * 64, k_end = min(D, (int)(blockIdx.x + 1) * length);
  float* dst = part + ((long)blockIdx.x * T + t0) * R;
  const Buffer rows_in = buffer_of(in + t0 * D, (uint32_t)count * D * 2u);
  for (int item = mine; item < units * (4 / NF); item += share) {  // first halves before second
    const int u = item < units ? item : item - units;
    const int start = uniform(lds.start[u]), end = uniform(lds.start[u + 1]);
    const int at = item < units ? start : start + 16 * NF, len = min(16 * NF, end - at);
    const int adapter = uniform(lds.key[start] >> 10);
    if (len <= 0 || adapter == n) continue;
    const int nf = (len + 15) >> 4;
    uint32_t x[2 * NF];  // where row 8 j + lane / 8 begins
#pragma unroll
    for (int j = 0; j < 2 * NF; ++j)
      x[j] = (lds.key[at + min(8 * j + row8, len - 1)] & (kSpan - 1)) * (uint32_t)D * 2u;
    const Buffer w = buffer_of(W + (long)adapter * R * D, (uint32_t)R * D * 2u);
    floatx4 acc[NF][NR];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int c = 0; c < NR; ++c) acc[f][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = k_begin; k0 < k_end; k0 += 64 * kWaves) {
      Block16 xb[NF];
      const int kc = k0 + 8 * chunk;
#pragma unroll
      for (int j = 0; j < 2 * NF; ++j)
        xb[j >> 1].load(j & 1, rows_in, x[j] + 2u * kc, 8 * j + row8 < len && kc < k_end);
      bf16x8_t wv[NR][2];
      if constexpr (kTrans) {
        Rows8<NR> rows[2];
        const int r0 = NR * col, k = k0 + 8 * g;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            rows[h].load(j, w, ((uint32_t)k * R + r0) * 2u, k + 32 * h < k_end && r0 < R, (32 * h + j) * R * 2);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          wv[c][0] = rows[0].column(c);
          wv[c][1] = rows[1].column(c);
        }
      } else {
        Block16 wb[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = NR * (8 * j + row8) + c;
            wb[c].load(j, w, ((uint32_t)r * D + kc) * 2u, r < R && kc < k_end);
          }
#pragma unroll
        for (int c = 0; c < NR; ++c) wb[c].turn(turn[wave][c & 1], lane, wv[c][0], wv[c][1]);
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if (f >= nf) continue;
        bf16x8_t lo, hi;
        xb[f].turn(turn[wave][f & 1], lane, lo, hi);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          acc[f][c] = mfma16(wv[c][0], lo, acc[f][c]);
          acc[f][c] = mfma16(wv[c][1], hi, acc[f][c]);
        }
      }
    }
    // the waves' sums, in wave order; value (c, lane, i) is r = 4 NR g + NR i + c
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      if (f >= nf) continue;
#pragma unroll
      for (int c = 0; c < NR; ++c) red[wave][c][lane] = acc[f][c];
      __syncthreads();
      const int m = 16 * f + col;
      for (int q = wave; q < NR; q += kWaves) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (4 * q + e) / NR, c = (4 * q + e) % NR;
          float sum = red[0][c][lane][i];
#pragma unroll
          for (int y = 1; y < kWaves; ++y) sum += red[y][c][lane][i];
          v[e] = sum;
        }
        const int r = 4 * NR * g + 4 * q;
        if (m < len && r < R) store_at<floatx4>(dst, (uint32_t)((at + m) * R + r) * 4u, v);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- expansion to N (or H)
// Two values as hi + lo in BF16, 16 significant bits each. What lies beyond BF16's largest value is
// left to lo (2^120 at most, or infinity), so that hi never rounds up to an infinity that lo would
// have to take back.
__device__ __forceinline__ float within_bf16(float x) {
  constexpr float kMost = 0x1.fep+127f;
  return __builtin_amdgcn_fmed3f(x, -kMost, kMost);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = f32x2_to_bf16x2(within_bf16(x), within_bf16(y));
  lo = f32x2_to_bf16x2(x - bf16_to_f32(hi & 0xFFFFu), y - bf16_to_f32(hi >> 16));
}

// Rows of the low-rank vectors of a unit in LDS: the sum of the parts (in
// order) times the adapter's scale, as hi and lo. With R <= 16 one row holds
// hi[16] lo[16], which fill the 32 k of one MFMA; with more, hi[] and lo[] are
// planes of whole steps of 32 that meet the same operand of the matrix.
template <int NR>
struct LowRows {
  static constexpr int kSteps = NR == 1 ? 1 : NR / 2;
  static constexpr int kLo = NR == 1 ? 16 : 32 * kSteps;  // where lo begins
  static constexpr int kStride = 2 * kLo + 8;
  uint16_t v[kUnit][kStride];
};

// Adds base to 16 FP32 columns of a token, c[0 .. 7] at `offset` and c[8 .. 15] 32 columns
// further, and stores them in BF16. Four lanes then write 64 bytes at a stretch.
__device__ __forceinline__ void store16(uint16_t* out, uint32_t offset, bool first, bool second,
                                        const float (&c)[16], const uint4 (&base)[2]) {
  uint32_t o[8];
  const uint32_t b[8] = {base[0].x, base[0].y, base[0].z, base[0].w, base[1].x, base[1].y, base[1].z, base[1].w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    o[j] = f32x2_to_bf16x2(bf16_to_f32(b[j] & 0xFFFFu) + c[2 * j], bf16_to_f32(b[j] >> 16) + c[2 * j + 1]);
  if (first) store_at<uint4>(out, offset, make_uint4(o[0], o[1], o[2], o[3]));
  if (second) store_at<uint4>(out, offset + 64u, make_uint4(o[4], o[5], o[6], o[7]));
}

// Columns, and threads, of an expanding workgroup. Each one adds the parts of its tokens again, so
// wide ones pay as soon as there are enough of them: T = 4096, n = 4, H = N = 7168, R = 128 takes 97
// us a call with 512 and 107 with 256, T = 8192, n = 6, R = 16 81.7 and 83.3; T = 2048, n = 8,
// H = N = 4096, R = 32 25.8 and 23.9.
static int expand_cols(int T, int D) { return (long)T * D >= 1l << 24 ? 512 : 256; }

// out[t][c] = bf16(base[t][c] + sum_r low[t][r] W_a[c][r]) (kTrans: W_a[r][c]),
// low = scale * (sum of the parts). blockIdx.x is a block of kCols columns, 64 for each wave,
// so that neighbouring workgroups write neighbouring pieces of the same tokens; blockIdx.y
// is a span and one of `share` workgroups that take its units in turn. Workgroups with
// blockIdx.x == 0 also write the sum of the parts to `sums` (times the scale if scale_sums),
// 0 without an adapter.
// Operand row i of block b is column 32 (b / 2) + 8 (i / 4) + 4 (b % 2) + i % 4, with kTrans
// 32 (i / 2 % 2) + 8 (i / 4) + 4 (i % 2) + b; either way a lane's four blocks end as the
// columns 8 g .. 8 g + 7 and 32 further of one token, so that four lanes read and write 64
// bytes at a stretch. With kTrans W_a has its columns contiguous while an operand wants eight
// r of one column: a lane reads four columns of eight rows and turns them in registers.
// Bound by HBM: T = 8192, n = 6, N = 7168, R = 16 takes 50 us, 235 MB at 4.7 TB/s. Fetching the
// next unit's rows ahead halved the waves that fit, and lost.
template <int NR, bool kTrans, int kCols>
__global__ __launch_bounds__(kCols) void adapter_expand_kernel(
    const float* __restrict__ part, int parts, const SpanOrder* __restrict__ orders, int share, int T,
    int D, int R, const uint16_t* __restrict__ W, const float* __restrict__ scale,
    const uint16_t* base, uint16_t* out, float* __restrict__ sums, int scale_sums) {
  using Low = LowRows<NR>;
  __shared__ __align__(16) Low low;
  __shared__ int place[kUnit];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int sp = blockIdx.y / share;
  const SpanOrder* order = orders + sp;
  const int units = order->units;
  const long t0 = (long)sp * kSpan;
  const int c0 = blockIdx.x * kCols + 64 * wave;
  const int c = c0 + 8 * g;  // the lane's columns of the result: c .. c + 7 and c + 32 .. c + 39
  // tokens without an adapter: base, or zeros
  const bool fill = out != nullptr && base != out;
  if (base) base += t0 * D;
  if (out) out += t0 * D;
  const Buffer base_rows = buffer_of(base, base ? (uint32_t)min((long)kSpan, T - t0) * D * 2u : 0u);
  const bool keep_sums = sums != nullptr && blockIdx.x == 0;
  if (sums) sums += t0 * R;
  part += t0 * R;
  for (int u = blockIdx.y % share; u < units; u += share) {
    const uint2 unit = order->unit[u];
    const int at = uniform(unit.x & 0xFFFFu), len = uniform(unit.x >> 16), adapter = uniform(unit.y);
    __syncthreads();  // the unit before is no longer read
    if (tid < kUnit) place[tid] = order->key[at + min(tid, len - 1)] & (kSpan - 1);
    if (adapter == kNone) {
      __syncthreads();
      if (fill)
        for (int m = tid / (kCols / 8); m < len; m += 8) {
          const int cn = blockIdx.x * kCols + tid % (kCols / 8) * 8;
          const uint32_t o = (place[m] * (uint32_t)D + cn) * 2u;
          if (cn < D) store_at<uint4>(out, o, base ? load_at<uint4>(base, o) : make_uint4(0, 0, 0, 0));
        }
      if (keep_sums)
        for (int i = tid; i < len * R; i += kCols) sums[place[i / R] * R + i % R] = 0.0f;
      continue;
    }
    const int nf = (len + 15) >> 4;
    const float s = scale[adapter];
    const Buffer w = buffer_of(W + (long)adapter * R * D, (uint32_t)R * D * 2u);
    bf16x8_t wop[Low::kSteps][4];
    if constexpr (kTrans) {
      Rows8<4> rows[Low::kSteps];
      const int cc = c0 + 8 * (col >> 2) + 4 * (col & 1) + 16 * (col & 2);
#pragma unroll
      for (int q = 0; q < Low::kSteps; ++q) {
        const int rg = NR == 1 ? 8 * (g & 1) : 8 * g;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          rows[q].load(j, w, ((uint32_t)rg * D + cc) * 2u, cc < D && 32 * q + rg < R, (32 * q + j) * D * 2);
      }
#pragma unroll
      for (int q = 0; q < Low::kSteps; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b) wop[q][b] = rows[q].column(b);
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int cc = c0 + 32 * (b >> 1) + 8 * (col >> 2) + 4 * (b & 1) + (col & 3);
#pragma unroll
        for (int q = 0; q < Low::kSteps; ++q) {
          const int r = NR == 1 ? 8 * (g & 1) : 32 * q + 8 * g;
          wop[q][b] = as_bf16x8(load_if<uint4>(w, ((uint32_t)cc * R + r) * 2u, cc < D && r < R));
        }
      }
    }
    __syncthreads();  // place
    uint4 bv[4][2];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * f + col;
      const uint32_t b = (place[m] * (uint32_t)D + c) * 2u;  // without base the buffer is empty
      bv[f][0] = load_if<uint4>(base_rows, b, m < len && c < D);
      bv[f][1] = load_if<uint4>(base_rows, b + 64u, m < len && c + 32 < D);
    }
#pragma unroll 1
    for (int i = tid; i < nf * 16 * (4 * NR); i += kCols) {
      const int m = i / (4 * NR), r = i % (4 * NR) * 4;
      floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (m < len && r < R) {
        const uint32_t o = (uint32_t)((at + m) * R + r) * 4u;
        for (int p = 0; p < parts; p += 4) {
          floatx4 q[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) q[y] = load_at<floatx4>(part + (long)min(p + y, parts - 1) * T * R, o);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (p + y < parts) v += q[y];
        }
        if (keep_sums) store_at<floatx4>(sums, (place[m] * (uint32_t)R + r) * 4u, scale_sums ? v * s : v);
      }
      uint2 hi, lo;
      split2(v[0] * s, v[1] * s, hi.x, lo.x);
      split2(v[2] * s, v[3] * s, hi.y, lo.y);
      *reinterpret_cast<uint2*>(&low.v[m][r]) = hi;
      *reinterpret_cast<uint2*>(&low.v[m][Low::kLo + r]) = lo;
    }
    __syncthreads();
    if (out == nullptr || c0 >= D) continue;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (f >= nf) continue;
      floatx4 acc[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      const uint16_t* row = low.v[16 * f + col];
#pragma unroll
      for (int q = 0; q < Low::kSteps; ++q) {
        const uint4 vh = *reinterpret_cast<const uint4*>(row + 32 * q + 8 * g);
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = mfma16(wop[q][b], as_bf16x8(vh), acc[b]);
        if (NR > 1) {
          const uint4 vl = *reinterpret_cast<const uint4*>(row + Low::kLo + 32 * q + 8 * g);
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[b] = mfma16(wop[q][b], as_bf16x8(vl), acc[b]);
        }
      }
      if (16 * f + col < len) {
        float res[16];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) res[kTrans ? 4 * i + b : 4 * b + i] = acc[b][i];
        store16(out, (place[16 * f + col] * (uint32_t)D + c) * 2u, c < D, c + 32 < D, res, bv[f]);
      }
    }
  }
}

// ---------------------------------------------------------------- gradients of the matrices
// Two values as h + m + l in BF16, exactly: h is the upper half of x, which holds its first 8
// significant bits, m that of the rest, and what then remains has 8 bits at most. An infinite
// value gives NaN.
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  constexpr uint32_t kUpper = 0x07060302u;  // {upper half of the first, upper half of the second}
  const auto upper = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); };
  h = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), kUpper);
  const float x1 = x - upper(x), y1 = y - upper(y);
  m = __builtin_amdgcn_perm(__float_as_uint(y1), __float_as_uint(x1), kUpper);
  const float x2 = x1 - upper(x1), y2 = y1 - upper(y1);
  l = __builtin_amdgcn_perm(__float_as_uint(y2), __float_as_uint(x2), kUpper);
}

constexpr int kWindow = 4096;  // tokens of one window, of which an adapter's are listed in LDS
constexpr int kShare = 512;    // listed tokens from which a window is shared by several workgroups
constexpr int kMostShares = 8;
__host__ __device__ inline int grad_windows(int T) { return T > kWindow ? (T + kWindow - 1) / kWindow : 1; }
// Columns of one workgroup of the gradient kernels: 128 with R <= 32 (adapter_grad_kernel),
// above 256 (adapter_grad_wide_kernel).
static int grad_cols(int R) { return R <= 32 ? 128 : 256; }

struct GradParams {
  const uint16_t* x;    // [T][H]
  const uint16_t* dy;   // [T][N]
  const float* du;      // [T][R], scaled
  const float* v;       // [T][R]
  const float* scale;   // [n]
  const void* ids;
  int ids64, T, n, H, N, R;
  int groups, most_shares;  // groups of windows, and shares of each
  float* d_down;        // [n][R][H]
  float* d_up;          // [n][N][R]
  float* part_down;     // sums of the shares [groups * most_shares][n][R][H], with more than one in all
  float* part_up;       // [groups * most_shares][n][N][R], likewise
  int* shares;          // [groups][n]: shares that were used, likewise
};

// What a workgroup of the gradient kernels works on: adapter blockIdx.y, kCols columns of x
// (dA) or, behind those, of dy (dB), kRows values of r from r_begin on, and a share
// (blockIdx.z % most_shares) of the adapter's tokens in each window of a group
// (blockIdx.z / most_shares). A window of 4096 tokens has as many shares as have 512 of the
// adapter's tokens each, but one at least and most_shares at most.
template <bool kDown>
struct GradBlock {
  int c0, r_begin, D, share, group;
  float scale;
  int used;               // most shares of a window so far
  // of the current window
  Buffer in;              // rows of x or dy, tokens count from the window's first
  Buffer low;             // rows of du or v
  int first, last;        // the share's places in the list

  __device__ __forceinline__ GradBlock(const GradParams& p, int kCols, int kRows) {
    const int down_chunks = (p.H + kCols - 1) / kCols;
    const int chunks = down_chunks + (p.N + kCols - 1) / kCols;
    const int chunk = blockIdx.x % chunks;
    r_begin = blockIdx.x / chunks * kRows;
    c0 = (kDown ? chunk : chunk - down_chunks) * kCols;
    D = kDown ? p.H : p.N;
    scale = kDown ? 1.0f : p.scale[blockIdx.y];
    group = blockIdx.z / p.most_shares;
    share = blockIdx.z % p.most_shares;
    used = group == 0 ? 1 : 0;  // the first leaves zeros where there are no tokens at all
  }

  // Windows of the group.
  __device__ __forceinline__ int begin(const GradParams& p) const {
    return (int)((long)grad_windows(p.T) * group / p.groups);
  }
  __device__ __forceinline__ int end(const GradParams& p) const {
    return (int)((long)grad_windows(p.T) * (group + 1) / p.groups);
  }

  // kThreads threads list the adapter's tokens of the window in order, thread t those among
  // the t-th kWindow / kThreads tokens; behind the share come 64 times -1. Begins and ends
  // with a barrier.
  template <int kThreads>
  __device__ __forceinline__ void list_window(const GradParams& p, int window, int* list, int* wave_count) {
    constexpr int kPer = kWindow / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, a = blockIdx.y;
    const long t0 = (long)window * kWindow;
    const int count = (int)min((long)kWindow, p.T - t0);
    uint32_t hit = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int t = tid * kPer + j;
      if (t < count && adapter_of(p.ids, p.ids64, t0 + t, p.n) == a) hit |= 1u << j;
    }
    const int incl = wave_inclusive_sum(__popc(hit));
    __syncthreads();  // the window before is done with
    if (lane == 63) wave_count[wave] = incl;
    __syncthreads();
    int at = incl - __popc(hit), have = 0;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) at += wave_count[w];
      have += wave_count[w];
    }
    have = uniform(have);
    const int shares = min((have + kShare - 1) / kShare, p.most_shares);
    const int each = shares > 0 ? ((have + shares - 1) / shares + 31) & ~31 : 0;
    first = min(share * each, have);
    last = share < shares ? min(first + each, have) : first;
    used = max(used, shares);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (hit >> j & 1) {
        if (at < last) list[at] = tid * kPer + j;
        ++at;
      }
    if (tid < 64) list[last + tid] = -1;
    in = buffer_of((kDown ? p.x : p.dy) + t0 * D, (uint32_t)count * D * 2u);
    low = buffer_of((kDown ? p.du : p.v) + t0 * p.R, (uint32_t)count * p.R * 4u);
    __syncthreads();
  }

  // Where the sums go: [R][H] or [N][R], null if the share was never used. The first
  // workgroup leaves the number of shares for adapter_sum_kernel.
  __device__ __forceinline__ float* output(const GradParams& p) const {
    const int a = blockIdx.y;
    if (p.groups * p.most_shares > 1 && share == 0 && blockIdx.x == 0 && threadIdx.x == 0)
      p.shares[group * p.n + a] = used;
    if (share >= used) return nullptr;
    const bool whole = p.groups == 1 && used == 1;
    float* to = kDown ? (whole ? p.d_down : p.part_down) : (whole ? p.d_up : p.part_up);
    return to + (whole ? a : (long)blockIdx.z * p.n + a) * p.R * D;
  }
};

// Whether a workgroup has columns of x.
__device__ __forceinline__ bool grad_down(const GradParams& p, int kCols) {
  const int down_chunks = (p.H + kCols - 1) / kCols;
  return (int)blockIdx.x % (down_chunks + (p.N + kCols - 1) / kCols) < down_chunks;
}

// Eight values of one column of du (s v), as the three operands of split3.
__device__ __forceinline__ void split3_column(const float (&v)[8], float s, uint4& h, uint4& m, uint4& l) {
  split3(v[0] * s, v[1] * s, h.x, m.x, l.x);
  split3(v[2] * s, v[3] * s, h.y, m.y, l.y);
  split3(v[4] * s, v[5] * s, h.z, m.z, l.z);
  split3(v[6] * s, v[7] * s, h.w, m.w, l.w);
}

// acc[b] += (columns of x) (r)^T, or for dB (r) (columns of dy)^T.
template <bool kDown, int NB>
__device__ __forceinline__ void grad_mfma(const bf16x8_t (&op)[NB], uint4 low, floatx4 (&acc)[NB]) {
  const bf16x8_t w = as_bf16x8(low);
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = kDown ? mfma16(op[b], w, acc[b]) : mfma16(w, op[b], acc[b]);
}

// The listed tokens of step k0 for lane group g, and their rows' columns.
template <bool kDown, int NB>
__device__ __forceinline__ void grad_fetch(const GradBlock<kDown>& q, const int* list, int k0, int g, int cc,
                                           int (&tok)[8], Rows8<NB>& rows) {
  const int4 a = *reinterpret_cast<const int4*>(&list[k0 + 8 * g]);
  const int4 b = *reinterpret_cast<const int4*>(&list[k0 + 8 * g + 4]);
  const int t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    tok[j] = t[j];
    rows.load(j, q.in, ((uint32_t)t[j] * q.D + cc) * 2u, t[j] >= 0 && cc < q.D);
  }
}
template <bool kDown>
__device__ __forceinline__ void grad_low(const GradBlock<kDown>& q, int R, const int (&tok)[8], int r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = load_if<float>(q.low, ((uint32_t)tok[j] * R + r) * 4u, tok[j] >= 0 && r < R);
}

// The gradients for R <= 32, 128 columns and all r to a workgroup of four waves, which take
// every fourth step of 32 tokens, the rows of the next step on their way during one. k is the
// token here, so both operands are wanted with eight tokens of one column: x (dy) is turned in
// registers, du (s v) is read column by column. Bound by the latency of that chain of list, rows
// and du, in which the list weighs most, for a thread waits for each of its 16 ids before it asks for
// the next: T = 1100, n = 6, H = 2064, N = 2688, R = 8 takes 12 us, where 9 MB are to be read (one
// token in seven has no adapter).
struct GradLds {
  int list[kWindow + 64];
  int wave_count[4];
  floatx4 red[4][8][64];
};
template <int NR, bool kDown>
__device__ __forceinline__ void grad_body(const GradParams& p, GradLds& lds) {
  constexpr int NB = 8, kCols = 16 * NB;
  int* list = lds.list;
  floatx4(*red)[NB][64] = lds.red;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4, R = p.R;
  GradBlock<kDown> q(p, kCols, 16 * NR);
  floatx4 acc[NR][NB];
#pragma unroll
  for (int c = 0; c < NR; ++c)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[c][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int cc = q.c0 + NB * col;
  const int end = q.end(p);
  for (int window = q.begin(p); window < end; ++window) {
    q.template list_window<256>(p, window, list, lds.wave_count);
    const int begin = q.first + 32 * wave;
    Rows8<NB> next;
    int tok[8];
    if (begin < q.last) grad_fetch(q, list, begin, g, cc, tok, next);
    for (int k0 = begin; k0 < q.last; k0 += 128) {
      bf16x8_t op[NB];
      float lv[NR][8];
#pragma unroll
      for (int c = 0; c < NR; ++c) grad_low(q, R, tok, 16 * c + col, lv[c]);
#pragma unroll
      for (int b = 0; b < NB; ++b) op[b] = next.column(b);
      if (k0 + 128 < q.last) grad_fetch(q, list, k0 + 128, g, cc, tok, next);
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        uint4 h, m, l;
        split3_column(lv[c], q.scale, h, m, l);
        grad_mfma<kDown>(op, l, acc[c]);
        grad_mfma<kDown>(op, m, acc[c]);
        grad_mfma<kDown>(op, h, acc[c]);
      }
    }
  }
  float* out = q.output(p);
  if (out == nullptr) return;
  // the waves' sums in wave order, 16 values of r at a time; the lanes' places in LDS are turned
  // by 4 g, so that the reads meet all banks
#pragma unroll
  for (int c = 0; c < NR; ++c) {
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][b][g * 16 + ((col + 4 * g) & 15)] = acc[c][b];
    __syncthreads();
    if constexpr (kDown) {
      // value (b, lane (col, g), i) is row r = 16 c + col, column c0 + NB (4 g + i) + b
      const int r16 = tid >> 4, gi = tid & 15, gg = gi >> 2;
      const int r = 16 * c + r16, h = q.c0 + NB * gi, ln = gg * 16 + ((r16 + 4 * gg) & 15);
#pragma unroll
      for (int o = 0; o < NB; o += 4) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = ((red[0][o + e][ln][gi & 3] + red[1][o + e][ln][gi & 3]) + red[2][o + e][ln][gi & 3]) +
                 red[3][o + e][ln][gi & 3];
        if (r < R && h < q.D) *reinterpret_cast<floatx4*>(out + (long)r * q.D + h + o) = v;
      }
    } else {
      // value (b, lane (col, g), i) is row c0 + NB col + b, column r = 16 c + 4 g + i
#pragma unroll
      for (int item = tid; item < kCols * 4; item += 256) {
        const int gg = item & 3, cl = item >> 2 & 15, b = item >> 6, row = NB * cl + b;
        const int ln = gg * 16 + ((cl + 4 * gg) & 15);
        const floatx4 v = ((red[0][b][ln] + red[1][b][ln]) + red[2][b][ln]) + red[3][b][ln];
        const int r = 16 * c + 4 * gg;
        if (r < R && q.c0 + row < q.D)
          *reinterpret_cast<floatx4*>(out + (long)(q.c0 + row) * R + r) = v;
      }
    }
    __syncthreads();
  }
}

template <int NR>
__global__ __launch_bounds__(256, NR == 1 ? 3 : 2) void adapter_grad_kernel(GradParams p) {
  __shared__ __align__(16) GradLds lds;
  if (grad_down(p, 128))
    grad_body<NR, true>(p, lds);
  else
    grad_body<NR, false>(p, lds);
}

// The gradients for R > 32: 256 columns and 64 values of r (with R > 64 there are two such
// halves) to a workgroup of eight waves. Four waves take 64 columns each of the even steps of
// 32 tokens, four of the odd ones. The three operands of du (s v), the same for all columns,
// are made once for the four: each wave reads and splits 16 of the 64 r and leaves them in
// LDS, in two buffers, so that one barrier a step is enough; it waits for LDS alone, the
// loads of the next step stay in flight. T = 4096, n = 4 runs of 1024, H = N = 7168, R = 64 takes
// 42 us: 22.5 GFLOP, three products to a factor, at 540 TFLOP/s (a large product: 1200), and 117 MB
// at 2.8 TB/s. Runs of random length, a fifth of the tokens without an adapter, take 51: the longest
// share decides. Each operand is waited for before its four products, and 14 registers are spilled.
// R = 17 .. 32 leaves half of its rows empty: T = 4096, n = 4, H = N = 7168, R = 32 takes 101 us a
// call with it and 88 with the kernel above.
struct GradWideLds {
  int list[kWindow + 64];
  int wave_count[8];
  // [buffer][even, odd][c][l, m, h][lane]; behind the loop the waves' sums [wave][b][lane]
  uint4 low[2][2][4][3][64];
};
template <bool kDown>
__device__ __forceinline__ void grad_wide_body(const GradParams& p, GradWideLds& lds) {
  constexpr int NR = 4, NB = 4, kCols = 64 * NB;
  int* list = lds.list;
  auto& low = lds.low;
  floatx4(*red)[NB][64] = reinterpret_cast<floatx4(*)[NB][64]>(lds.low);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4, part = wave & 3, odd = wave >> 2, R = p.R;
  GradBlock<kDown> q(p, kCols, 16 * NR);
  floatx4 acc[NR][NB];
#pragma unroll
  for (int c = 0; c < NR; ++c)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[c][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int cc = q.c0 + 16 * NB * part + NB * col;
  const int r_mine = q.r_begin + 16 * part + col;
  const int end = q.end(p);
  for (int window = q.begin(p); window < end; ++window) {
    q.template list_window<512>(p, window, list, lds.wave_count);
    Rows8<NB> next;
    int tok[8];
    float lv[8];
    // both halves take the same number of steps; behind the share lie 64 times -1
    if (q.first < q.last) {
      grad_fetch(q, list, q.first + 32 * odd, g, cc, tok, next);
      grad_low(q, R, tok, r_mine, lv);
    }
    int buffer = 0;
    for (int k0 = q.first; k0 < q.last; k0 += 64) {
      uint4 h, m, l;
      split3_column(lv, q.scale, h, m, l);
      low[buffer][odd][part][0][lane] = l;
      low[buffer][odd][part][1][lane] = m;
      low[buffer][odd][part][2][lane] = h;
      bf16x8_t op[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) op[b] = next.column(b);
      if (k0 + 64 < q.last) {
        grad_fetch(q, list, k0 + 64 + 32 * odd, g, cc, tok, next);
        grad_low(q, R, tok, r_mine, lv);
      }
      lds_barrier();
#pragma unroll
      for (int c = 0; c < NR; ++c)
#pragma unroll
        for (int y = 0; y < 3; ++y) {
          grad_mfma<kDown>(op, low[buffer][odd][c][y][lane], acc[c]);
          __builtin_amdgcn_sched_barrier(0);  // else all twelve operands are held at once: spills
        }
      buffer ^= 1;
    }
  }
  float* out = q.output(p);
  if (out == nullptr) return;
#pragma unroll
  for (int c = 0; c < NR; ++c) {
    __syncthreads();  // the operands, or the sums before, are no longer read
    // the lanes' places are turned by 4 (w % 4) + g, so that the reads meet all banks
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][b][g * 16 + ((col + 4 * part + g) & 15)] = acc[c][b];
    __syncthreads();
    if constexpr (kDown) {
      // value (b, lane (col, g), i) of wave w is row r = r_begin + 16 c + col, column
      // c0 + 64 (w % 4) + 4 (4 g + i) + b
#pragma unroll
      for (int item = tid; item < 16 * kCols / 4; item += 512) {
        const int r16 = item >> 6, w = item >> 4 & 3, gi = item & 15, gg = gi >> 2;
        const int ln = gg * 16 + ((r16 + 4 * w + gg) & 15);
        const int r = q.r_begin + 16 * c + r16, h = q.c0 + 64 * w + 4 * gi;
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = red[w][e][ln][gi & 3] + red[w + 4][e][ln][gi & 3];
        if (r < R && h < q.D) *reinterpret_cast<floatx4*>(out + (long)r * q.D + h) = v;
      }
    } else {
      // value (b, lane (col, g), i) of wave w is row c0 + 64 (w % 4) + 4 col + b, column
      // r = r_begin + 16 c + 4 g + i
#pragma unroll
      for (int item = tid; item < kCols * 4; item += 512) {
        const int gg = item & 3, cl = item >> 2 & 15, b = item >> 6 & 3, w = item >> 8, row = 64 * w + 4 * cl + b;
        const int ln = gg * 16 + ((cl + 4 * w + gg) & 15);
        const floatx4 v = red[w][b][ln] + red[w + 4][b][ln];
        const int r = q.r_begin + 16 * c + 4 * gg;
        if (r < R && q.c0 + row < q.D)
          *reinterpret_cast<floatx4*>(out + (long)(q.c0 + row) * R + r) = v;
      }
    }
  }
}

__global__ __launch_bounds__(512, 4) void adapter_grad_wide_kernel(GradParams p) {
  __shared__ __align__(16) GradWideLds lds;
  if (grad_down(p, 256))
    grad_wide_body<true>(p, lds);
  else
    grad_wide_body<false>(p, lds);
}

// Adds the shares of the groups, in order, where there is more than one in all: quads
// [0, na4) of the adapter's [R][H], then those of its [N][R]. Adapter blockIdx.y.
__global__ __launch_bounds__(256) void adapter_sum_kernel(GradParams p) {
  const int a = blockIdx.y;
  if (p.groups == 1 && p.shares[a] == 1) return;  // written in place
  const long na4 = (long)p.R * p.H / 4, nb4 = (long)p.R * p.N / 4;
  for (long i = blockIdx.x * 256L + threadIdx.x; i < na4 + nb4; i += (long)gridDim.x * 256) {
    const bool first = i < na4;
    const long size = first ? na4 : nb4, k = a * size + (first ? i : i - na4);
    const floatx4* part = reinterpret_cast<const floatx4*>(first ? p.part_down : p.part_up) + k;
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int y = 0; y < p.groups; ++y) {
      const int shares = p.shares[y * p.n + a];
      for (int s = 0; s < shares; ++s) v += part[(long)(y * p.most_shares + s) * p.n * size];
    }
    reinterpret_cast<floatx4*>(first ? p.d_down : p.d_up)[k] = v;
  }
}

// ---------------------------------------------------------------- launches
#define PMOE_BY_RANK(R, call)   \
  do {                          \
    if ((R) <= 16) {            \
      constexpr int NR = 1;     \
      call;                     \
    } else if ((R) <= 32) {     \
      constexpr int NR = 2;     \
      call;                     \
    } else if ((R) <= 64) {     \
      constexpr int NR = 4;     \
      call;                     \
    } else {                    \
      constexpr int NR = 8;     \
      call;                     \
    }                           \
  } while (0)

static int spans_of(int T) { return (T + kSpan - 1) / kSpan; }

// Workgroups that share the units of a span: as many as there can be while the launch stays
// within some thousand workgroups.
static int span_share(int T, int n, int others) {
  const int tokens = T < kSpan ? T : kSpan;
  const int most = (tokens + kUnit - 1) / kUnit + (n < tokens ? n : tokens);
  const int room = 8192 / (spans_of(T) * others);
  return room < 1 ? 1 : (room < most ? room : most);
}

namespace {
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The workspace: the orders of the spans, the parts of the reduction, and for the backward
// call du and the sums of the shares.
struct AdapterLayout {
  SpanOrder* orders;
  float *part, *du, *part_down, *part_up;
  int* shares;
  size_t bytes;
};
}  // namespace

// Groups of windows and shares of a window: as many as it takes to fill the GPU where few
// adapters make few workgroups. More workgroups cost more than they bring, for each has to list
// its tokens and leaves sums to be added: T = 4096, n = 4, H = N = 7168 took 88 us a call with 256
// and 104 with 1024 wanted (R = 32), 125 with 512, 130 with 768 and 132 with 256 (R = 64).
struct GradSplit {
  int groups, shares;
};
static GradSplit grad_split(int T, int n, int H, int N, int R) {
  const int cols = grad_cols(R), windows = grad_windows(T);
  const long each = (long)n * ((H + cols - 1) / cols + (N + cols - 1) / cols) * (R > 64 ? 2 : 1);
  const int want = (int)(((R <= 32 ? 256 : 512) + each - 1) / each);
  GradSplit g;
  g.groups = windows < want ? windows : want;
  g.shares = (want + g.groups - 1) / g.groups;
  const int most = T < kWindow ? (T + kShare - 1) / kShare : kMostShares;
  if (g.shares > most) g.shares = most;
  if (g.shares < 1) g.shares = 1;
  return g;
}

static AdapterLayout adapter_layout(void* ws, int T, int n, int H, int N, int R, bool backward) {
  AdapterLayout l;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    char* at = static_cast<char*>(ws) + o;
    o += up256(bytes);
    return at;
  };
  l.orders = reinterpret_cast<SpanOrder*>(take(sizeof(SpanOrder) * spans_of(T)));
  l.part = reinterpret_cast<float*>(take((size_t)adapter_parts(backward ? N : H, R) * T * R * 4));
  if (backward) {
    const GradSplit g = grad_split(T, n, H, N, R);
    const int slots = g.groups * g.shares;
    const size_t each = slots > 1 ? (size_t)slots * n * R * 4 : 0;
    l.du = reinterpret_cast<float*>(take((size_t)T * R * 4));
    l.part_down = reinterpret_cast<float*>(take(each * H));
    l.part_up = reinterpret_cast<float*>(take(each * N));
    l.shares = reinterpret_cast<int*>(take((size_t)g.groups * n * 4));
  }
  l.bytes = o;
  return l;
}

static hipError_t reduce(bool trans, const void* in, const AdapterParams& p, int D, const void* W,
                         const AdapterLayout& l, hipStream_t s) {
  const int parts = adapter_parts(D, p.R), share = span_share(p.T, p.n, parts);
  const dim3 grid(parts, spans_of(p.T) * share);
  const int length = adapter_part_length(D, p.R);
  const uint16_t* x = static_cast<const uint16_t*>(in);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  if (trans)
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, true><<<grid, 64 * reduce_waves(p.R), 0, s>>>(
                          x, p.ids, p.ids64, p.T, p.n, D, p.R, w, length, share, l.orders, l.part)));
  else
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, false><<<grid, 64 * reduce_waves(p.R), 0, s>>>(
                          x, p.ids, p.ids64, p.T, p.n, D, p.R, w, length, share, l.orders, l.part)));
  return hipGetLastError();
}

template <bool kTrans, int kCols>
static hipError_t expand_by(int parts, const AdapterParams& p, int D, const void* W, const AdapterLayout& l,
                            float* sums, int scale_sums, hipStream_t s) {
  const int chunks = p.out ? (D + kCols - 1) / kCols : 1, share = span_share(p.T, p.n, chunks);
  const dim3 grid(chunks, spans_of(p.T) * share);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const uint16_t* b = static_cast<const uint16_t*>(p.base);
  uint16_t* o = static_cast<uint16_t*>(p.out);
  PMOE_BY_RANK(p.R, (adapter_expand_kernel<NR, kTrans, kCols><<<grid, kCols, 0, s>>>(
                        l.part, parts, l.orders, share, p.T, D, p.R, w, p.scale, b, o, sums, scale_sums)));
  return hipGetLastError();
}

template <bool kTrans>
static hipError_t expand(int parts, const AdapterParams& p, int D, const void* W, const AdapterLayout& l,
                         float* sums, int scale_sums, hipStream_t s) {
  return expand_cols(p.T, D) == 512 ? expand_by<kTrans, 512>(parts, p, D, W, l, sums, scale_sums, s)
                                    : expand_by<kTrans, 256>(parts, p, D, W, l, sums, scale_sums, s);
}

size_t adapter_forward_ws_bytes(int T, int n, int H, int N, int R) {
  return adapter_layout(nullptr, T, n, H, N, R, false).bytes;
}

size_t adapter_backward_ws_bytes(int T, int n, int H, int N, int R) {
  return adapter_layout(nullptr, T, n, H, N, R, true).bytes;
}

hipError_t launch_adapter_forward(const AdapterParams& p, hipStream_t s) {
  const AdapterLayout l = adapter_layout(p.ws, p.T, p.n, p.H, p.N, p.R, false);
  const hipError_t e = reduce(false, p.x, p, p.H, p.down, l, s);
  if (e != hipSuccess) return e;
  return expand<false>(adapter_parts(p.H, p.R), p, p.N, p.up, l, p.v_out, 0, s);
}

hipError_t launch_adapter_backward(const AdapterParams& p, hipStream_t s) {
  const AdapterLayout l = adapter_layout(p.ws, p.T, p.n, p.H, p.N, p.R, true);
  if (p.T > 0) {
    hipError_t e = reduce(true, p.dy, p, p.N, p.up, l, s);
    if (e != hipSuccess) return e;
    e = expand<true>(adapter_parts(p.N, p.R), p, p.H, p.down, l, l.du, 1, s);
    if (e != hipSuccess) return e;
  }
  if (!p.d_down) return hipSuccess;
  GradParams q;
  q.x = static_cast<const uint16_t*>(p.x);
  q.dy = static_cast<const uint16_t*>(p.dy);
  q.du = l.du;
  q.v = p.v_in;
  q.scale = p.scale;
  q.ids = p.ids;
  q.ids64 = p.ids64;
  q.T = p.T, q.n = p.n, q.H = p.H, q.N = p.N, q.R = p.R;
  const GradSplit split = grad_split(p.T, p.n, p.H, p.N, p.R);
  q.groups = split.groups, q.most_shares = split.shares;
  q.d_down = p.d_down, q.d_up = p.d_up;
  q.part_down = l.part_down, q.part_up = l.part_up, q.shares = l.shares;
  const int cols = grad_cols(p.R), chunks = (p.H + cols - 1) / cols + (p.N + cols - 1) / cols;
  const dim3 grid(chunks * (p.R > 64 ? 2 : 1), p.n, q.groups * q.most_shares);
  if (p.R <= 16)
    adapter_grad_kernel<1><<<grid, 256, 0, s>>>(q);
  else if (p.R <= 32)
    adapter_grad_kernel<2><<<grid, 256, 0, s>>>(q);
  else
    adapter_grad_wide_kernel<<<grid, 512, 0, s>>>(q);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || q.groups * q.most_shares == 1) return e;
  const long quads = (long)p.R * (p.H + p.N) / 4, blocks = (quads + 255) / 256, room = 8192 / p.n + 1;
  adapter_sum_kernel<<<dim3((int)(blocks < room ? blocks : room), p.n), 256, 0, s>>>(q);
  return hipGetLastError();
}

}  // namespace pmoe

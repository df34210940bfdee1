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
// bits), three (24 bits, all of FP32) where it stays FP32.
#include "device.h"
#include "kernels.h"

namespace pmoe {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 64;    // tokens of one unit at most
constexpr int kSpan = 1024;  // tokens that are grouped together
constexpr int kNone = -1;  // adapter of a unit of tokens without one
constexpr int kMostRuns = 16;  // boundaries up to which a span is not sorted

__device__ __forceinline__ floatx4 mfma16(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Loads and stores at a 32-bit byte offset from a pointer that is the same in all lanes: the
// pointer stays in scalar registers. Offsets within a span of tokens or within one adapter's
// matrix, and within a segment of 4096 tokens, are at most 2^27.
template <typename V>
__device__ __forceinline__ V load_at(const void* base, uint32_t offset) {
  return *reinterpret_cast<const V*>(static_cast<const char*>(base) + offset);
}
template <typename V>
__device__ __forceinline__ void store_at(void* base, uint32_t offset, V v) {
  *reinterpret_cast<V*>(static_cast<char*>(base) + offset) = v;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 u) { return __builtin_bit_cast(bf16x8_t, u); }

__device__ __forceinline__ int adapter_of(const void* ids, int ids64, long t, int n) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[t] : static_cast<const int*>(ids)[t];
  return id >= 0 && id < n ? (int)id : -1;
}

constexpr int kReduceWaves = 8;
constexpr int kReduceThreads = 64 * kReduceWaves;

// Order and units of a span: unit u holds the places [start[u], start[u + 1]) of
// the order; key = adapter << 10 | token of the span, adapter n for none.
constexpr int kChunks = kSpan / 64;
struct SpanLds {
  uint32_t key[kSpan];
  uint16_t start[kSpan + 8];
  int table[16][kChunks];  // sort: keys of a digit in a chunk of 64, then the places before them
  int wave[2][kReduceWaves];
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

// Groups the tokens [t0, t0 + count) with a workgroup of kReduceThreads; returns
// the number of units. Ends with a barrier.
__device__ __forceinline__ int group_span(const void* ids, int ids64, long t0, int count, int n, SpanLds& l) {
  constexpr int kPer = kSpan / kReduceThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid + kReduceThreads * j;
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
    const int i = tid + kReduceThreads * j;
    edges += __popcll(__ballot(i > 0 && i < count && key[j] >> 10 != l.key[max(i, 1) - 1] >> 10));
  }
  if (lane == 0) l.wave[0][wave] = edges;
  __syncthreads();
  edges = 0;
  for (int w = 0; w < kReduceWaves; ++w) edges += l.wave[0][w];
  if (edges > kMostRuns) {
    // Stable sort by adapter, four bits at a time from the lowest: a key's place is the number of
    // keys with a smaller digit, plus those with its digit in the chunks before its own, plus
    // those among the lanes below (found by ballots on the digit's bits).
    const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
    for (int shift = 10; n >> (shift - 10) != 0; shift += 4) {
      for (int i = tid; i < 16 * kChunks; i += kReduceThreads) (&l.table[0][0])[i] = 0;
      __syncthreads();
      int digit[kPer], rank[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool on = tid + kReduceThreads * j < count;
        digit[j] = key[j] >> shift & 15;
        uint64_t match = __ballot(on);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint64_t set = __ballot(digit[j] >> b & 1);
          match &= digit[j] >> b & 1 ? set : ~set;
        }
        rank[j] = __popcll(match & below);
        if (on && rank[j] == 0) l.table[digit[j]][wave + kReduceWaves * j] = __popcll(match);
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
        if (tid + kReduceThreads * j < count)
          l.key[l.table[digit[j]][wave + kReduceWaves * j] + rank[j]] = key[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] = l.key[tid + kReduceThreads * j];
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
  for (int w = 0; w < kReduceWaves; ++w) {
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

__device__ __forceinline__ void keep_order(const SpanLds& l, int units, int count, int n, SpanOrder* o) {
  for (int i = threadIdx.x; i < count; i += kReduceThreads) o->key[i] = l.key[i];
  for (int i = threadIdx.x; i < units; i += kReduceThreads) {
    const uint32_t at = l.start[i], len = l.start[i + 1] - at;
    const int a = l.key[at] >> 10;
    o->unit[i] = make_uint2(at | len << 16, a == n ? kNone : a);
  }
  if (threadIdx.x == 0) o->units = units;
}

// ---------------------------------------------------------------- reduction over H (or N)
// A sum over a row of D elements is cut into parts of adapter_part_length(D) elements (a
// multiple of 64, at most 2048), one workgroup of eight waves each, whose waves take pieces of
// 64 elements in turn: together they read a row in long stretches.
int adapter_parts(int D) { return (D + 2047) / 2048; }
static int adapter_part_length(int D) { return ((D + adapter_parts(D) - 1) / adapter_parts(D) + 63) / 64 * 64; }

// Eight rows of kCols columns each, turned: op[b] gets the eight values of
// column b, ready as an MFMA operand. kCols is 1, 2, 4 or 8.
template <int kCols>
struct Rows8 {
  static constexpr int kWords = kCols < 2 ? 1 : kCols / 2;
  uint32_t w[8][kWords];
  __device__ __forceinline__ void load(int j, const void* base, uint32_t offset, bool on) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[j][i] = 0;
    if (!on) return;
    if constexpr (kCols == 1) {
      w[j][0] = load_at<uint16_t>(base, offset);
    } else if constexpr (kCols == 2) {
      w[j][0] = load_at<uint32_t>(base, offset);
    } else if constexpr (kCols == 4) {
      const uint2 u = load_at<uint2>(base, offset);
      w[j][0] = u.x, w[j][1] = u.y;
    } else {
      const uint4 u = load_at<uint4>(base, offset);
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
  __device__ __forceinline__ void load(int j, const void* base, uint32_t offset, bool on) {
    v[j] = make_uint4(0, 0, 0, 0);
    if (on) v[j] = load_at<uint4>(base, offset);
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
template <int NR, bool kTrans>
__global__ __launch_bounds__(kReduceThreads, NR <= 2 ? 4 : 2) void adapter_reduce_kernel(
    const uint16_t* __restrict__ in, const void* __restrict__ ids, int ids64, int T, int n, int D, int R,
    const uint16_t* __restrict__ W, int length, int share, SpanOrder* __restrict__ orders,
    float* __restrict__ part) {
  constexpr int NF = NR <= 4 ? 4 : 2;      // row blocks of an item: a unit, or half a unit
  __shared__ __align__(16) SpanLds lds;
  __shared__ uint4 turn[kReduceWaves][2][128];
  __shared__ floatx4 red[kReduceWaves][NR][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4, row8 = lane >> 3, chunk = lane & 7;
  const int sp = blockIdx.y / share, mine = blockIdx.y % share;
  const long t0 = (long)sp * kSpan;
  const int count = (int)min((long)kSpan, T - t0);
  const int units = group_span(ids, ids64, t0, count, n, lds);
  if (mine == 0 && blockIdx.x == 0) keep_order(lds, units, count, n, orders + sp);
  const int k_begin = blockIdx.x * length + wave * 64, k_end = min(D, (int)(blockIdx.x + 1) * length);
  float* dst = part + ((long)blockIdx.x * T + t0) * R;
  const uint16_t* rows_in = in + t0 * D;
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
    const uint16_t* w = W + (long)adapter * R * D;
    floatx4 acc[NF][NR];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int c = 0; c < NR; ++c) acc[f][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = k_begin; k0 < k_end; k0 += 64 * kReduceWaves) {
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
            rows[h].load(j, w + (32 * h + j) * R, ((uint32_t)k * R + r0) * 2u, k + 32 * h < k_end && r0 < R);
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
      for (int q = wave; q < NR; q += kReduceWaves) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (4 * q + e) / NR, c = (4 * q + e) % NR;
          float sum = red[0][c][lane][i];
#pragma unroll
          for (int y = 1; y < kReduceWaves; ++y) sum += red[y][c][lane][i];
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
// Two values as hi + lo in BF16, 16 significant bits each. An infinite value has lo = 0.
__device__ __forceinline__ float finite_rest(float x, float hi) {
  return __builtin_fabsf(x) == __builtin_inff() ? 0.0f : x - hi;
}
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = f32x2_to_bf16x2(x, y);
  lo = f32x2_to_bf16x2(finite_rest(x, bf16_to_f32(hi & 0xFFFFu)), finite_rest(y, bf16_to_f32(hi >> 16)));
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

// out[t][c] = bf16(base[t][c] + sum_r low[t][r] W_a[c][r]) (kTrans: W_a[r][c]),
// low = scale * (sum of the parts). blockIdx.x is a block of 256 columns, 64 for each wave,
// so that neighbouring workgroups write neighbouring pieces of the same tokens; blockIdx.y
// is a span and one of `share` workgroups that take its units in turn. Workgroups with
// blockIdx.x == 0 also write the sum of the parts to `sums` (times the scale if scale_sums),
// 0 without an adapter.
// Operand row i of block b is column 32 (b / 2) + 8 (i / 4) + 4 (b % 2) + i % 4, with kTrans
// 32 (i / 2 % 2) + 8 (i / 4) + 4 (i % 2) + b; either way a lane's four blocks end as the
// columns 8 g .. 8 g + 7 and 32 further of one token, so that four lanes read and write 64
// bytes at a stretch. With kTrans W_a has its columns contiguous while an operand wants eight
// r of one column: a lane reads four columns of eight rows and turns them in registers.
template <int NR, bool kTrans>
__global__ __launch_bounds__(256) void adapter_expand_kernel(
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
  const int c0 = blockIdx.x * 256 + 64 * wave;
  const int c = c0 + 8 * g;  // the lane's columns of the result: c .. c + 7 and c + 32 .. c + 39
  // tokens without an adapter: base, or zeros
  const bool fill = out != nullptr && base != out;
  if (base) base += t0 * D;
  if (out) out += t0 * D;
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
        for (int m = tid >> 5; m < len; m += 8) {
          const int cn = blockIdx.x * 256 + (tid & 31) * 8;
          const uint32_t o = (place[m] * (uint32_t)D + cn) * 2u;
          if (cn < D) store_at<uint4>(out, o, base ? load_at<uint4>(base, o) : make_uint4(0, 0, 0, 0));
        }
      if (keep_sums)
        for (int i = tid; i < len * R; i += 256) sums[place[i / R] * R + i % R] = 0.0f;
      continue;
    }
    const int nf = (len + 15) >> 4;
    const float s = scale[adapter];
    const uint16_t* w = W + (long)adapter * R * D;
    bf16x8_t wop[Low::kSteps][4];
    if constexpr (kTrans) {
      Rows8<4> rows[Low::kSteps];
      const int cc = c0 + 8 * (col >> 2) + 4 * (col & 1) + 16 * (col & 2);
#pragma unroll
      for (int q = 0; q < Low::kSteps; ++q) {
        const int rg = NR == 1 ? 8 * (g & 1) : 8 * g;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          rows[q].load(j, w + (long)(32 * q + j) * D, ((uint32_t)rg * D + cc) * 2u, cc < D && 32 * q + rg < R);
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
          uint4 v = make_uint4(0, 0, 0, 0);
          if (cc < D && r < R) v = load_at<uint4>(w, ((uint32_t)cc * R + r) * 2u);
          wop[q][b] = as_bf16x8(v);
        }
      }
    }
    __syncthreads();  // place
    uint4 bv[4][2];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      bv[f][0] = bv[f][1] = make_uint4(0, 0, 0, 0);
      if (f < nf && base && 16 * f + col < len) {
        const uint32_t b = (place[16 * f + col] * (uint32_t)D + c) * 2u;
        if (c < D) bv[f][0] = load_at<uint4>(base, b);
        if (c + 32 < D) bv[f][1] = load_at<uint4>(base, b + 64u);
      }
    }
#pragma unroll 1
    for (int i = tid; i < nf * 16 * (4 * NR); i += 256) {
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
// Two values as h + m + l in BF16: all 24 bits of an FP32 value. An infinite value has
// m = l = 0.
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = f32x2_to_bf16x2(x, y);
  const float x1 = finite_rest(x, bf16_to_f32(h & 0xFFFFu)), y1 = finite_rest(y, bf16_to_f32(h >> 16));
  m = f32x2_to_bf16x2(x1, y1);
  l = f32x2_to_bf16x2(x1 - bf16_to_f32(m & 0xFFFFu), y1 - bf16_to_f32(m >> 16));
}

constexpr int kSegMax = 4096;  // tokens of one segment at most; an adapter's are listed in LDS
// Columns of one workgroup of adapter_grad_kernel, 16 NB: with R <= 32 NB = 8, above (where
// there are four blocks of r) NB = 4, so that the accumulators leave room for two waves.
static int grad_cols(int R) { return R <= 32 ? 128 : 64; }

struct GradParams {
  const uint16_t* x;    // [T][H]
  const uint16_t* dy;   // [T][N]
  const float* du;      // [T][R], scaled
  const float* v;       // [T][R]
  const float* scale;   // [n]
  const void* ids;
  int ids64, T, n, H, N, R, seg;
  float* d_down;        // [n][R][H], or with several segments the partial sums [segments][n][R][H]
  float* d_up;          // [n][N][R], likewise
};

// One workgroup: adapter blockIdx.y, segment blockIdx.z, 16 NB columns of x (dA)
// or, behind those, of dy (dB), and 16 NR values of r (with R > 64 there are two
// such halves). The
// adapter's tokens of the segment are listed in LDS, the waves take every fourth
// step of 32 of them, the rows of the next step on their way during one. k is the
// token here, so both operands are wanted with eight tokens of one column: x (dy)
// is turned in registers, du (s v) is read column by column.
template <int NR, int NB>
__global__ __launch_bounds__(256, 2) void adapter_grad_kernel(GradParams p) {
  __shared__ __align__(16) int list[kSegMax + 32];
  __shared__ int wave_count[4];
  __shared__ floatx4 red[4][NB][64];
  constexpr int kCols = 16 * NB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int a = blockIdx.y, seg0 = blockIdx.z * p.seg;
  const int seg1 = min(p.T, seg0 + p.seg);
  const int down_chunks = (p.H + kCols - 1) / kCols;
  const int chunks = down_chunks + (p.N + kCols - 1) / kCols;
  const int chunk = blockIdx.x % chunks, r_begin = blockIdx.x / chunks * (16 * NR);
  const bool down = chunk < down_chunks;
  const int c0 = (down ? chunk : chunk - down_chunks) * kCols;
  const int D = down ? p.H : p.N, R = p.R;
  const uint16_t* in = (down ? p.x : p.dy) + (long)seg0 * D;  // tokens count from the segment's first
  const float* low = (down ? p.du : p.v) + (long)seg0 * R;
  const float s = down ? 1.0f : p.scale[a];
  // the adapter's tokens, in order: thread t looks at the t-th 16 of the segment
  uint32_t hit = 0;
#pragma unroll
  for (int j = 0; j < kSegMax / 256; ++j) {
    const int t = seg0 + tid * (kSegMax / 256) + j;
    if (t < seg1 && adapter_of(p.ids, p.ids64, t, p.n) == a) hit |= 1u << j;
  }
  const int incl = wave_inclusive_sum(__popc(hit));
  if (lane == 63) wave_count[wave] = incl;
  __syncthreads();
  int at = incl - __popc(hit), have = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) at += wave_count[w];
    have += wave_count[w];
  }
#pragma unroll
  for (int j = 0; j < kSegMax / 256; ++j)
    if (hit >> j & 1) list[at++] = tid * (kSegMax / 256) + j;
  if (tid < 32) list[have + tid] = -1;
  __syncthreads();
  floatx4 acc[NR][NB];
#pragma unroll
  for (int c = 0; c < NR; ++c)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[c][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int cc = c0 + NB * col;
  Rows8<NB> next;
  int tok[8];
  const auto fetch = [&](int k0) {
    const int4 t0 = *reinterpret_cast<const int4*>(&list[k0 + 8 * g]);
    const int4 t1 = *reinterpret_cast<const int4*>(&list[k0 + 8 * g + 4]);
    const int t[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      tok[j] = t[j];
      next.load(j, in, ((uint32_t)t[j] * D + cc) * 2u, t[j] >= 0 && cc < D);
    }
  };
  if (32 * wave < have) fetch(32 * wave);
  for (int k0 = 32 * wave; k0 < have; k0 += 128) {
    bf16x8_t op[NB];
    float lv[NR][8];
#pragma unroll
    for (int c = 0; c < NR; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r_begin + 16 * c + col;
        lv[c][j] = tok[j] >= 0 && r < R ? load_at<float>(low, ((uint32_t)tok[j] * R + r) * 4u) : 0.0f;
      }
#pragma unroll
    for (int b = 0; b < NB; ++b) op[b] = next.column(b);
    if (k0 + 128 < have) fetch(k0 + 128);
#pragma unroll
    for (int c = 0; c < NR; ++c) {
      uint32_t h[4], m[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split3(lv[c][2 * j] * s, lv[c][2 * j + 1] * s, h[j], m[j], l[j]);
      const bf16x8_t ho = as_bf16x8(make_uint4(h[0], h[1], h[2], h[3]));
      const bf16x8_t mo = as_bf16x8(make_uint4(m[0], m[1], m[2], m[3]));
      const bf16x8_t lo = as_bf16x8(make_uint4(l[0], l[1], l[2], l[3]));
      if (down) {  // rows: columns of x, columns: r
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(op[b], lo, acc[c][b]);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(op[b], mo, acc[c][b]);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(op[b], ho, acc[c][b]);
      } else {     // rows: r, columns: columns of dy
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(lo, op[b], acc[c][b]);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(mo, op[b], acc[c][b]);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[c][b] = mfma16(ho, op[b], acc[c][b]);
      }
    }
  }
  // the waves' sums in wave order, 16 values of r at a time
  const long slot = (long)blockIdx.z * p.n + a;
#pragma unroll
  for (int c = 0; c < NR; ++c) {
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][b][lane] = acc[c][b];
    __syncthreads();
    if (down) {
      // value (b, lane (col, g), i) is row r = r_begin + 16 c + col, column c0 + NB (4 g + i) + b
      const int r16 = tid >> 4, gi = tid & 15;
      const int r = r_begin + 16 * c + r16, h = c0 + NB * gi, ln = (gi >> 2) * 16 + r16;
#pragma unroll
      for (int q = 0; q < NB; q += 4) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = ((red[0][q + e][ln][gi & 3] + red[1][q + e][ln][gi & 3]) + red[2][q + e][ln][gi & 3]) +
                 red[3][q + e][ln][gi & 3];
        if (r < R && h < D) *reinterpret_cast<floatx4*>(p.d_down + (slot * R + r) * D + h + q) = v;
      }
    } else {
      // value (b, lane (col, g), i) is row c0 + NB col + b, column r = r_begin + 16 c + 4 g + i
#pragma unroll
      for (int item = tid; item < kCols * 4; item += 256) {
        const int row = item >> 2, gg = item & 3, b = row % NB, ln = gg * 16 + row / NB;
        const floatx4 v = ((red[0][b][ln] + red[1][b][ln]) + red[2][b][ln]) + red[3][b][ln];
        const int r = r_begin + 16 * c + 4 * gg;
        if (r < R && c0 + row < D) *reinterpret_cast<floatx4*>(p.d_up + (slot * D + c0 + row) * R + r) = v;
      }
    }
    __syncthreads();
  }
}

// Sums over the segments, in order, for both gradients: quads [0, na4) of the one, then nb4
// of the other.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const floatx4* __restrict__ pa, const floatx4* __restrict__ pb,
                                                          int segments, long na4, long nb4,
                                                          floatx4* __restrict__ oa, floatx4* __restrict__ ob) {
  for (long i = blockIdx.x * 256L + threadIdx.x; i < na4 + nb4; i += (long)gridDim.x * 256) {
    const bool first = i < na4;
    const long k = first ? i : i - na4, stride = first ? na4 : nb4;
    const floatx4* part = (first ? pa : pb) + k;
    floatx4 v = part[0];
#pragma unroll 4
    for (int s = 1; s < segments; ++s) v += part[s * stride];
    (first ? oa : ob)[k] = v;
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
// call du and the segments' gradients.
struct AdapterLayout {
  SpanOrder* orders;
  float *part, *du, *d_down, *d_up;
  size_t bytes;
};
}  // namespace

static int grad_segment(int T, int n, int H, int N, int R);

static AdapterLayout adapter_layout(void* ws, int T, int n, int H, int N, int R, bool backward) {
  AdapterLayout l;
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    char* at = static_cast<char*>(ws) + o;
    o += up256(bytes);
    return at;
  };
  l.orders = reinterpret_cast<SpanOrder*>(take(sizeof(SpanOrder) * spans_of(T)));
  l.part = reinterpret_cast<float*>(take((size_t)adapter_parts(backward ? N : H) * T * R * 4));
  if (backward) {
    const int seg = grad_segment(T, n, H, N, R), segments = (T + seg - 1) / seg;
    const size_t each = segments > 1 ? (size_t)segments * n * R * 4 : 0;
    l.du = reinterpret_cast<float*>(take((size_t)T * R * 4));
    l.d_down = reinterpret_cast<float*>(take(each * H));
    l.d_up = reinterpret_cast<float*>(take(each * N));
  }
  l.bytes = o;
  return l;
}

static hipError_t reduce(bool trans, const void* in, const AdapterParams& p, int D, const void* W,
                         const AdapterLayout& l, hipStream_t s) {
  const int parts = adapter_parts(D), share = span_share(p.T, p.n, parts);
  const dim3 grid(parts, spans_of(p.T) * share);
  const int length = adapter_part_length(D);
  const uint16_t* x = static_cast<const uint16_t*>(in);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  if (trans)
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, true><<<grid, kReduceThreads, 0, s>>>(
                          x, p.ids, p.ids64, p.T, p.n, D, p.R, w, length, share, l.orders, l.part)));
  else
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, false><<<grid, kReduceThreads, 0, s>>>(
                          x, p.ids, p.ids64, p.T, p.n, D, p.R, w, length, share, l.orders, l.part)));
  return hipGetLastError();
}

static hipError_t expand(bool trans, int parts, const AdapterParams& p, int D, const void* W,
                         const AdapterLayout& l, float* sums, int scale_sums, hipStream_t s) {
  const int chunks = p.out ? (D + 255) / 256 : 1, share = span_share(p.T, p.n, chunks);
  const dim3 grid(chunks, spans_of(p.T) * share);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const uint16_t* b = static_cast<const uint16_t*>(p.base);
  uint16_t* o = static_cast<uint16_t*>(p.out);
  if (trans)
    PMOE_BY_RANK(p.R, (adapter_expand_kernel<NR, true><<<grid, 256, 0, s>>>(
                          l.part, parts, l.orders, share, p.T, D, p.R, w, p.scale, b, o, sums, scale_sums)));
  else
    PMOE_BY_RANK(p.R, (adapter_expand_kernel<NR, false><<<grid, 256, 0, s>>>(
                          l.part, parts, l.orders, share, p.T, D, p.R, w, p.scale, b, o, sums, scale_sums)));
  return hipGetLastError();
}

// Segments of the tokens for the gradients of the matrices: several where few adapters make few
// workgroups.
static int grad_segment(int T, int n, int H, int N, int R) {
  const int cols = grad_cols(R);
  const long per_segment = (long)n * ((H + cols - 1) / cols + (N + cols - 1) / cols);
  int seg = kSegMax;
  while (seg > 512 && per_segment * ((T + seg - 1) / seg) < 384) seg /= 2;
  return seg;
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
  return expand(false, adapter_parts(p.H), p, p.N, p.up, l, p.v_out, 0, s);
}

hipError_t launch_adapter_backward(const AdapterParams& p, hipStream_t s) {
  const AdapterLayout l = adapter_layout(p.ws, p.T, p.n, p.H, p.N, p.R, true);
  if (p.T > 0) {
    hipError_t e = reduce(true, p.dy, p, p.N, p.up, l, s);
    if (e != hipSuccess) return e;
    e = expand(true, adapter_parts(p.N), p, p.H, p.down, l, l.du, 1, s);
    if (e != hipSuccess) return e;
  }
  if (!p.d_down) return hipSuccess;
  const int seg = grad_segment(p.T, p.n, p.H, p.N, p.R);
  const int segments = p.T > 0 ? (p.T + seg - 1) / seg : 1;
  GradParams q;
  q.x = static_cast<const uint16_t*>(p.x);
  q.dy = static_cast<const uint16_t*>(p.dy);
  q.du = l.du;
  q.v = p.v_in;
  q.scale = p.scale;
  q.ids = p.ids;
  q.ids64 = p.ids64;
  q.T = p.T, q.n = p.n, q.H = p.H, q.N = p.N, q.R = p.R, q.seg = seg;
  q.d_down = segments > 1 ? l.d_down : p.d_down;
  q.d_up = segments > 1 ? l.d_up : p.d_up;
  const int cols = grad_cols(p.R), chunks = (p.H + cols - 1) / cols + (p.N + cols - 1) / cols;
  const dim3 grid(chunks * (p.R > 64 ? 2 : 1), p.n, segments);
  PMOE_BY_RANK(p.R, (adapter_grad_kernel<(NR < 4 ? NR : 4), (NR < 4 ? 8 : 4)><<<grid, 256, 0, s>>>(q)));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || segments == 1) return e;
  const long na4 = (long)p.n * p.R * p.H / 4, nb4 = (long)p.n * p.R * p.N / 4;
  const long blocks = (na4 + nb4 + 255) / 256;
  adapter_sum_kernel<<<(int)(blocks < 8192 ? blocks : 8192), 256, 0, s>>>(
      reinterpret_cast<const floatx4*>(l.d_down), reinterpret_cast<const floatx4*>(l.d_up), segments, na4, nb4,
      reinterpret_cast<floatx4*>(p.d_down), reinterpret_cast<floatx4*>(p.d_up));
  return hipGetLastError();
}

}  // namespace pmoe

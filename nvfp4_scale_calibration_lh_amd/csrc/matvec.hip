// Products of a few rows with NVFP4 weights as the scale sweep leaves them, dense or per expert:
//   Y[t, c] = g * sum_k E2M1(nibble[c, k]) * E4M3(code[c, k / 16]) * x[t, k],
//   g = fp32(amax / (6 * norm)), for the rows t of each group against that group's matrix;
//   x is bf16, fp32, or E4M3 bytes times a scale per row or per 128 channels of a row.
//
// Bound by reading the weights once (0.5625 bytes each), so the layout is the one they are stored
// in: a lane reads 16 bytes (32 elements, two blocks) of one output channel, 16 channels by 128
// elements a wave, as the A operand of 16x16x32 matrix instructions whose columns are the rows of x
// (k in any order, as long as both operands have the same).  The waves of a workgroup share k among
// them and add their sums in LDS in a fixed order.
//
// 12288x4096: one bf16 row 9.3 us, sixteen E4M3 rows 11 us, 32 bf16 rows 19 us, 64 44 us; 4096x12288 with five fp32
// rows 16.5 us; 2048x2048 with one row 4.4 us traced; 320 bf16 rows over 512 experts of 1280x2560, 135 of them
// hit, 77 us (242 MB, 3.1 TB/s); 98304x4096 with one row 50 us (4.5 TB/s).  Reading the weights alone in
// this pattern takes 5.5 us at 12288x4096 (4.6 TB/s).
//
// E2M1 * E4M3 has at most 6 significant bits, so it is exact in bf16 (bf16 and fp32 x) and, its
// range being [2^-10, 2688], in fp16 (E4M3 x, also exact in fp16).  fp32 x is split into three
// bf16 pieces, exactly from 2^-110 on; a smaller x loses its bits under 2^-133, the smallest bf16 number (the
// matrix instructions take subnormal numbers).  Every product is exact; sums are fp32.
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v4u_a8 __attribute__((ext_vector_type(4), aligned(8)));   // rows are 8-byte aligned
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v2u_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned v4u_a1 __attribute__((ext_vector_type(4), aligned(1)));

constexpr int kChunk = 128;                  // elements of k a wave takes at a time
constexpr int kMaxWaves = 8;
constexpr int kComputeUnits = 256;

enum { kXBf16 = 0, kXF32 = 1, kXE4m3 = 2 };

struct Args {
  const void* x;
  const float* x_scale;
  const uint8_t* code;
  const uint8_t* fp4;
  const float* amax;
  const int64_t* offsets;
  void* y;
  int64_t rows, n_groups;
  int cout, cin, x_scales;                   // x_scales: scales of one row (1, or cin / 128 rounded up)
  float gdiv;
  int run;                                   // channel tiles of one workgroup
};

template <int X>
struct Frag {
  using type = b8;
  static constexpr int pieces = 1;
};
template <>
struct Frag<kXF32> {
  using type = b8;
  static constexpr int pieces = 3;
};
template <>
struct Frag<kXE4m3> {
  using type = h8;
  static constexpr int pieces = 1;
};

template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// Eight weights: the nibbles of word w times the E4M3 scale in byte B (0 or 2) of `code`.
template <int X, int B>
__device__ inline typename Frag<X>::type weights(unsigned w, unsigned code) {
  typename Frag<X>::type out;
  if constexpr (X == kXE4m3) {
    const h2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)code, 1.0f, B == 2);
    const h2 s = {s2[0], s2[0]};
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, P) * s;
      out[2 * P] = v[0];
      out[2 * P + 1] = v[1];
    });
  } else {
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)code, B);
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, P);
      const b2 r = __builtin_convertvector((v2f){v[0] * s, v[1] * s}, b2);   // exact
      out[2 * P] = r[0];
      out[2 * P + 1] = r[1];
    });
  }
  return out;
}

// Which elements of a chunk a lane multiplies at step S (8 of the 32 that an instruction takes).  A
// lane loads 32 neighbouring weights, element 8 * (4 * quarter + word).  Their words are exchanged
// between the quarters of the wave so that a load of x covers whole runs of a row, 64 bytes over the
// four quarters, where it would otherwise touch four runs (16 rows of bf16 took 4 times the cycles
// of the vector memory path, 10 us of 20 at 12288x4096):
//   bf16, fp32: both bits of the quarter against both of the word; element 8 * (4 * S + quarter)
//   E4M3: the quarter's high bit against the word's high bit, so a lane's 16 bytes of x are two words:
//         element 64 * (S / 2) + 32 * (quarter % 2) + 16 * (quarter / 2) + 8 * (S % 2)
template <int X>
__device__ inline v4u exchange(v4u w) {
  auto swap32 = [](unsigned& a, unsigned& b) {       // a's upper half of the wave against b's lower half
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  auto swap16 = [](unsigned& a, unsigned& b) {       // a's odd quarters against b's even quarters
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
  };
  unsigned n0 = w[0], n1 = w[1], n2 = w[2], n3 = w[3];
  swap32(n0, n2);
  swap32(n1, n3);
  if constexpr (X != kXE4m3) {
    swap16(n0, n1);
    swap16(n2, n3);
  }
  return v4u{n0, n1, n2, n3};
}
// The scale bytes of a lane's words 0, 1 (in bytes 0 and 2 of the first) and 2, 3, from a chunk's 8.
template <int X>
__device__ inline v2u lane_codes(v2u c, int quarter) {
  if constexpr (X == kXE4m3) {                       // words 0, 1 are one block of the first four, 2, 3 of the others
    const int by = 8 * (2 * (quarter & 1) + (quarter >> 1));
    return v2u{c[0] >> by, c[1] >> by};
  } else {                                           // word S is block 2 * S + quarter / 2
    const int by = 8 * (quarter >> 1);
    return v2u{c[0] >> by, c[1] >> by};
  }
}

// A lane's elements of x of one chunk, as loaded, and where load j starts.
template <int X>
struct Raw {
  static constexpr int per = X == kXF32 ? 4 : (X == kXBf16 ? 8 : 16);   // elements of 16 bytes
  v4u v[32 / per];
};
template <int X>
__device__ inline int first_of(int j, int quarter) {
  if (X == kXE4m3) return 64 * j + 32 * (quarter & 1) + 16 * (quarter >> 1);
  if (X == kXBf16) return 32 * j + 8 * quarter;
  return 32 * (j / 2) + 8 * quarter + 4 * (j % 2);
}
// Step S (8 elements) of it as matrix operands.
template <int X, int S>
__device__ inline void frag_x(const Raw<X>& r, typename Frag<X>::type* f) {
  if constexpr (X == kXBf16) {
    f[0] = __builtin_bit_cast(b8, r.v[S]);
  } else if constexpr (X == kXE4m3) {
    each<4>([&](auto pp) {
      constexpr int P = decltype(pp)::value;
      const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.v[S / 2][2 * (S % 2) + P / 2], 1.0f, P % 2 == 1);
      f[0][2 * P] = v[0];
      f[0][2 * P + 1] = v[1];
    });
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {                    // truncated pieces: 8 + 8 + 8 bits
      const float x = __uint_as_float(r.v[2 * S + e / 4][e % 4]);
      const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
      const float r1 = x == hi ? 0.0f : x - hi;      // an infinity is its first piece, not infinity minus infinity
      const float mid = __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
      f[0][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(hi) >> 16));
      f[1][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(mid) >> 16));
      f[2][e] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(r1 - mid) >> 16));
    }
  }
}

__device__ inline v4f mfma(b8 a, b8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ inline v4f mfma(h8 a, h8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ inline int64_t uniform(int64_t v) {       // the same on every lane, kept in scalar registers
  return (int64_t)((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)((uint64_t)v >> 32)) << 32 |
                   (unsigned)__builtin_amdgcn_readfirstlane((int)v));
}

// The piece-th run of at most `tile` rows of one group, over all groups in order: its group and
// rows, or group -1 past the last.  Every wave finds it by itself, without a barrier: 512 groups at a
// time, 8 neighbouring ones a lane.
struct Piece {
  int64_t group, row, rows;
};
__device__ inline Piece find_piece(const Args& a, unsigned piece, int tile) {
  if (a.n_groups == 1) {
    const int64_t row = (int64_t)piece * tile;
    return {row < a.rows ? 0 : -1, row, min((int64_t)tile, a.rows - row)};
  }
  constexpr int kEach = 8;
  const int lane = threadIdx.x & 63;
  unsigned before = 0;                               // pieces of the groups before this round's
  for (int64_t g0 = 0; g0 < a.n_groups; g0 += 64 * kEach) {
    const int64_t g = g0 + lane * kEach;
    int64_t off[kEach + 1];
#pragma unroll
    for (int k = 0; k <= kEach; ++k)                 // past the last group: empty ones
      off[k] = min(max(a.offsets[min(g + k, a.n_groups)], (int64_t)0), a.rows);
    unsigned n[kEach], mine = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) mine += n[k] = (unsigned)((max(off[k + 1] - off[k], (int64_t)0) + tile - 1) / tile);
    unsigned upto = mine;                            // inclusive scan over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    const unsigned all = __shfl(upto, 63, 64);
    if (piece - before < all) {                      // the same on every lane
      unsigned at = piece - before - (upto - mine);  // from this lane's first piece
      const int owner = __ffsll((unsigned long long)__ballot(piece - before < upto)) - 1;
      int64_t group = -1, row = 0, rows = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (group < 0 && at < n[k]) {
          group = g + k;
          row = off[k] + (int64_t)at * tile;
          rows = min((int64_t)tile, off[k + 1] - row);
        }
        at -= n[k];                                  // wraps below zero once the group is found
      }
      return {__shfl(group, owner, 64), __shfl(row, owner, 64), __shfl(rows, owner, 64)};
    }
    before += all;
  }
  return {-1, 0, 0};
}

// A lane's weights of one chunk of one channel tile, as loaded: 32 nibbles and the chunk's 8 scale bytes.
struct Weights {
  v4u nib;
  v2u code;
};

// X: type of x.  MT: 16-row tiles of x a workgroup takes.  NT: 16-channel tiles of the output it takes
// at a time, `run` times in a row.  U: chunks of k a wave takes at a time, so waves * U chunks a step.
// P: a piece has at most 16 / P rows, so the 16 columns of an instruction hold those rows of x for P
// neighbouring chunks: a chunk's products are right in its own columns of an accumulator of its own,
// and a wave loads, converts and keeps 1 / P of what 16 rows would take.
// FULL: there are whole chunks (cin >= 128).  D: steps whose weights are held or on their way (one being multiplied, D - 1 in flight): a compute
// unit needs some 40 KB in flight to keep its share of the memory's rate.
// KEEP: one step covers k, and a wave keeps its elements of x as matrix operands over all its tiles;
// otherwise it loads them at each step.  GT: tiles whose sums meet in LDS together.
// Rows past the last repeat it, as do channels: a column of the products depends on its own row alone
// and is not stored, and repeating costs no mask.  Everything that is the same over a wave (chunk,
// tile, base addresses) is kept scalar: at few rows the kernel is close to bound by issuing instructions.
template <int X, int MT, int NT, int U, int P, int D, bool KEEP, bool FULL, int GT>
__global__ __launch_bounds__(64 * kMaxWaves) void k_matvec(const Args a) {
  constexpr int kPieces = Frag<X>::pieces;
  constexpr unsigned kSize = X == kXF32 ? 4 : (X == kXBf16 ? 2 : 1);
  using frag = typename Frag<X>::type;
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kCols = 16 / P, kSets = U / P;        // rows of x in a column set; sets of chunks that share registers
  static_assert(U % P == 0 && (P == 1 || MT == 1), "column sets are whole");
  const int i = lane & 15, quarter = lane >> 4, pack = i / kCols;
  const int tiles = (a.cout + 16 * NT - 1) / (16 * NT), runs = (tiles + a.run - 1) / a.run;
  Piece pc = find_piece(a, blockIdx.x / (unsigned)runs, 16 * MT / P);
  pc = {uniform(pc.group), uniform(pc.row), uniform(pc.rows)};
  if (pc.group < 0) return;
  const int tile0 = (int)(blockIdx.x % (unsigned)runs) * a.run, tile1 = min(tile0 + a.run, tiles);

  const unsigned row_bytes = (unsigned)a.cin / 2, row_codes = (unsigned)a.cin / 16;
  const uint8_t* x = (const uint8_t*)a.x + pc.row * a.cin * kSize;
  const float* xs = X == kXE4m3 ? a.x_scale + pc.row * a.x_scales : nullptr;
  unsigned x_at[MT], xs_at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const unsigned r = min(16 * m + i % kCols, (int)pc.rows - 1);
    x_at[m] = (r * (unsigned)a.cin + first_of<X>(0, quarter)) * kSize;
    xs_at[m] = X == kXE4m3 ? r * (unsigned)a.x_scales : 0;
  }
  const int full = a.cin / kChunk, stride = waves * U;
  const int steps = KEEP ? 1 : max((full + stride - 1) / stride, 1);

  const int total = (tile1 - tile0) * steps;
  // A wave's U chunks of a step are neighbours, so one load takes the scale bytes of two and a row's
  // 128-byte lines are used whole.  Near the end of k they start earlier, and those that the wave
  // before has are left out (the caller's U is at most the number of whole chunks).
  auto first_chunk = [&](int step) { return min(step * stride + wave * U, full - U); };
  Weights w[D][U][NT];
  // the weights of the n-th step of this workgroup
  auto load_w = [&](Weights (&w)[U][NT], int n) __attribute__((always_inline)) {
    n = min(n, total - 1);                           // past the end: the last step again, so that the loads
    const int tile = tile0 + (KEEP ? n : n / steps);   // in flight are the same number on every path
    const int first = first_chunk(KEEP ? 0 : n % steps);
    const int c0 = tile * (16 * NT);
    const int64_t at = pc.group * a.cout + c0;
    const uint8_t* nib = a.fp4 + at * row_bytes + (size_t)first * (kChunk / 2);
    const uint8_t* code = a.code + at * row_codes + (size_t)first * (kChunk / 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const unsigned c = min(16 * n + i, a.cout - 1 - c0);
      const unsigned w_at = c * row_bytes + quarter * 16, c_at = c * row_codes;
#pragma unroll
      for (int u = 0; u < U; ++u) w[u][n].nib = *(const v4u_a8*)(nib + w_at + u * (kChunk / 2));
#pragma unroll
      for (int u = 0; u + 1 < U; u += 2) {
        const v4u_a1 v = *(const v4u_a1*)(code + c_at + u * (kChunk / 16));
        w[u][n].code = v2u{v[0], v[1]}, w[u + 1][n].code = v2u{v[2], v[3]};
      }
      if constexpr (U % 2 == 1) w[U - 1][n].code = *(const v2u_a1*)(code + c_at + (U - 1) * (kChunk / 16));
    }
  };
  // x is loaded a step ahead like the weights where the registers hold both
  constexpr bool AHEAD = !KEEP && X != kXF32 && MT <= 2;
  constexpr int kXSlots = AHEAD ? D : 1;
  Raw<X> raws[kXSlots][kSets][MT];
  float scales[kXSlots][kSets][MT];
  auto load_rows = [&](Raw<X> (&raw)[kSets][MT], float (&scale)[kSets][MT], int n) __attribute__((always_inline)) {
    const int first = first_chunk(KEEP ? 0 : min(n, total - 1) % steps);
#pragma unroll
    for (int u = 0; u < kSets; ++u) {
      const int c = first + u * P;
      const uint8_t* p = x + (size_t)c * (kChunk * kSize);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const unsigned at = x_at[m] + (P > 1 ? pack * (kChunk * kSize) : 0);
#pragma unroll
        for (int j = 0; j < 32 / Raw<X>::per; ++j) raw[u][m].v[j] = *(const v4u*)(p + at + first_of<X>(j, 0) * kSize);
        if constexpr (X == kXE4m3) scale[u][m] = xs[(size_t)(a.x_scales > 1 ? c + (P > 1 ? pack : 0) : 0) + xs_at[m]];
      }
    }
  };
  v4f accs[GT][NT][MT];
  // One chunk; rows(S, m, f) gives step S of row tile m.
  auto multiply = [&](v4f (&acc)[NT][MT], const Weights (&w)[NT], auto&& rows, const float (&scale)[MT]) __attribute__((always_inline)) {
    v4f part[NT][MT];
    if constexpr (X == kXE4m3) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[n][m] = v4f{0, 0, 0, 0};
    }
    auto& sum = *(X == kXE4m3 ? &part : &acc);
    v4u nibs[NT];
    v2u codes[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) nibs[n] = exchange<X>(w[n].nib), codes[n] = lane_codes<X>(w[n].code, quarter);
    each<4>([&](auto st) __attribute__((always_inline)) {
      constexpr int S = decltype(st)::value;
      frag fx[MT][kPieces];
#pragma unroll
      for (int m = 0; m < MT; ++m) rows(st, m, fx[m]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const auto fw = weights<X, X == kXE4m3 ? 0 : 2 * (S % 2)>(nibs[n][S], codes[n][S / 2]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < kPieces; ++p) sum[n][m] = mfma(fw, fx[m][p], sum[n][m]);
      }
    });
    if constexpr (X == kXE4m3) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] += scale[m] * part[n][m];
    }
  };

  const float g = a.amax[pc.group] / a.gdiv;
  extern __shared__ float red[];
  frag kept[KEEP ? kSets : 1][MT][4][kPieces];
  if constexpr (KEEP && FULL) load_rows(raws[0], scales[0], 0);
  if constexpr (FULL) {
#pragma unroll
    for (int d = 0; d < D - 1; ++d) {
      if constexpr (AHEAD) load_rows(raws[d], scales[d], d);
      load_w(w[d], d);
    }
  }
  if constexpr (KEEP && FULL) {
#pragma unroll
    for (int u = 0; u < kSets; ++u)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        each<4>([&](auto st) __attribute__((always_inline)) { frag_x<X, decltype(st)::value>(raws[0][u][m], kept[u][m][decltype(st)::value]); });
  }
  auto clear = [&](v4f (&acc)[NT][MT]) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0, 0, 0, 0};
  };
#pragma unroll
  for (int t = 0; t < GT; ++t) clear(accs[t]);
  // one step with the weights in slot `at`; the slot before it, just used up, is filled again
  auto one = [&](int n, v4f (&acc)[NT][MT], Weights (&at)[U][NT], Weights (&used)[U][NT], auto slot) __attribute__((always_inline)) {
    constexpr int kNow = AHEAD ? decltype(slot)::value : 0, kNext = (kNow + D - 1) % kXSlots;
    auto& raw = raws[kNow];
    auto& scale = scales[kNow];
    const int tile = tile0 + (KEEP ? n : n / steps), step = KEEP ? 0 : n % steps;
    const int mine = step * stride + wave * U, first = FULL ? first_chunk(step) : 0;
    if constexpr (FULL) {
      if constexpr (!KEEP) load_rows(raws[kNext], scales[kNext], AHEAD ? n + D - 1 : n);
      load_w(used, n + D - 1);
      v4f own[P][NT][MT];                              // of each column set
#pragma unroll
      for (int p = 0; p < P; ++p) clear(own[p]);
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        frag made[KEEP || P == 1 ? 1 : 4][MT][kPieces];
        if constexpr (!KEEP && P > 1) {                // once for the set's P chunks
#pragma unroll
          for (int m = 0; m < MT; ++m) each<4>([&](auto st) __attribute__((always_inline)) { frag_x<X, decltype(st)::value>(raw[s][m], made[decltype(st)::value][m]); });
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int u = s * P + p;
          if (first + u < mine) continue;
          multiply(P == 1 ? acc : own[p], at[u], [&](auto st, int m, frag* f) __attribute__((always_inline)) {
            constexpr int S = decltype(st)::value;
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
              if constexpr (KEEP) f[q] = kept[s][m][S][q];
              else if constexpr (P > 1) f[q] = made[S][m][q];
            }
            if constexpr (!KEEP && P == 1) frag_x<X, S>(raw[s][m], f);
          }, scale[s]);
        }
      }
      if constexpr (P > 1) {                           // each column from its own set
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          v4f v = own[0][n][0];
#pragma unroll
          for (int p = 1; p < P; ++p)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = pack >= p ? own[p][n][0][r] : v[r];
          acc[n][0] += v;
        }
      }
    }
    if (step + 1 < steps) return;                              // the short chunk comes with the last step
    if (full * kChunk < a.cin && wave == full % waves) {       // the last, short chunk: 16 elements at a time
      const int left = a.cin - full * kChunk, own = left - quarter * 32;
      const int c0 = tile * (16 * NT);
      const int64_t base = pc.group * a.cout + c0;
      Weights wt[NT];
      Raw<X> rt[MT];
      float st[MT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t c = base + min(16 * n + i, a.cout - 1 - c0);
        const uint8_t* pn = a.fp4 + c * row_bytes + (full * (kChunk / 2) + quarter * 16);
        const uint8_t* pq = a.code + c * row_codes + full * (kChunk / 16);
        wt[n].nib = v4u{0, 0, 0, 0};
        wt[n].code = v2u{0, 0};
        if (own >= 16) {
          const v2u v = *(const v2u*)pn;
          wt[n].nib[0] = v[0], wt[n].nib[1] = v[1];
        }
        if (own >= 32) {
          const v2u v = *(const v2u*)(pn + 8);
          wt[n].nib[2] = v[0], wt[n].nib[3] = v[1];
        }
#pragma unroll
        for (int b = 0; b < 7; ++b)
          if (16 * b < left) wt[n].code[b / 4] |= (unsigned)pq[b] << (8 * (b % 4));
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int j = 0; j < 32 / Raw<X>::per; ++j)
          rt[m].v[j] = first_of<X>(j, quarter) < left
                           ? *(const v4u*)(x + (size_t)full * (kChunk * kSize) + x_at[m] + first_of<X>(j, 0) * kSize)
                           : v4u{0, 0, 0, 0};
        if constexpr (X == kXE4m3) st[m] = xs[(size_t)(a.x_scales > 1 ? full : 0) + xs_at[m]];
      }
      auto rows = [&](auto at, int m, frag* f) __attribute__((always_inline)) { frag_x<X, decltype(at)::value>(rt[m], f); };
      if constexpr (P == 1) {
        multiply(acc, wt, rows, st);
      } else {                                         // in the first column set
        v4f part[NT][MT];
        clear(part);
        multiply(part, wt, rows, st);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[n][0][r] += pack == 0 ? part[n][0][r] : 0.0f;
      }
    }
  };
  // The waves' sums of `count` tiles from `tile` on, in the waves' order: a lane holds channels
  // 4 * quarter + r of row i of each 16x16 part.
  auto reduce = [&](int tile, int count) __attribute__((always_inline)) {
    const int size = GT * NT * MT * 256;
#pragma unroll
    for (int t = 0; t < GT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int part = (t * NT + n) * MT + m;
#pragma unroll
          for (int r = 0; r < 4; ++r) red[wave * size + (part * 4 + r) * 64 + lane] = accs[t][n][m][r];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * NT * count * (int)pc.rows; e += blockDim.x) {
      const int c = e % 16, row = e / 16 % (int)pc.rows, tn = e / (16 * (int)pc.rows), channel = (tile * NT + tn) * 16 + c;
      const float* from = red + (tn * MT + row / 16) * 256 + (c % 4) * 64 + (c / 4) * 16 + row % 16;
      float s = 0.0f;
      int v = 0;
      constexpr int kTogether = 8 / P;               // independent loads
      for (; v + kTogether <= waves; v += kTogether) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = from[(v + k / P) * size + k % P * kCols];
#pragma unroll
        for (int k = 0; k < 8; ++k) s += t[k];
      }
      for (; v < waves; ++v)
#pragma unroll
        for (int p = 0; p < P; ++p) s += from[v * size + p * kCols];
      if (channel >= a.cout) continue;
      const int64_t to = (pc.row + row) * a.cout + channel;
      if constexpr (X == kXF32)
        ((float*)a.y)[to] = s * g;
      else
        ((__bf16*)a.y)[to] = (__bf16)(s * g);
    }
    if (tile + GT < tile1) __syncthreads();          // the sums have been read
#pragma unroll
    for (int t = 0; t < GT; ++t) clear(accs[t]);
  };
  static_assert(KEEP || GT == 1, "tiles are counted in steps");
  if constexpr (GT == 1) {
    for (int n = 0; n < total; n += D)
      each<D>([&](auto dd) __attribute__((always_inline)) {
        constexpr int d = decltype(dd)::value;
        if (n + d < total) {
          one(n + d, accs[0], w[d], w[(d + D - 1) % D], dd);
          if ((n + d + 1) % steps == 0) reduce(tile0 + (n + d) / steps, 1);
        }
      });
  } else {
    static_assert(GT % D == 0, "slots repeat with the tiles");
    for (int n = 0; n < total; n += GT) {
      each<GT>([&](auto dd) __attribute__((always_inline)) {
        constexpr int d = decltype(dd)::value;
        if (n + d < total) one(n + d, accs[d], w[d % D], w[(d + D - 1) % D], dd);
      });
      reduce(tile0 + n, min(GT, total - n));
    }
  }
}

// Tiles of one workgroup: as many as leave about the waves that fit a compute unit's registers.
template <int X, int MT, int NT, int U, int P>
hipError_t launch_tile(Args a, hipStream_t stream) {
  constexpr int kTogether = 4;
  const int rows = 16 * MT / P, chunks = std::max(a.cin / kChunk, 1), tiles = (a.cout + 16 * NT - 1) / (16 * NT);
  const int steps = (chunks + kMaxWaves * U - 1) / (kMaxWaves * U);
  const int waves = (chunks + U * steps - 1) / (U * steps);
  const int64_t pieces = a.n_groups == 1 ? (a.rows + rows - 1) / rows : a.rows / rows + std::min(a.n_groups, a.rows);
  const int64_t resident = kComputeUnits * std::max((U <= 2 ? 16 : 8) / waves, 1) * (a.n_groups == 1 ? 1 : 4);
  // 8 tiles were better than 4 or 16 for one large matrix, 16 than 8 or 32 for several (more fetch the rows of x less
  // often, fewer even out better): 512 experts of 1280x2560 with 320 rows 75 us against 89 and 85, 384 of 1536x2560 with
  // 256 76, 82, 86, 256 of 2048x2048 with 512 81, 92, 83, 128 of 4096x1024 with 256 53, 60, 52.  Four times the
  // workgroups that are resident were better than twice or eight times that for 256 of 1280x2560 with 64 rows
  // (28 us, 33, 31) and within 4% of the best elsewhere.
  a.run = (int)std::min<int64_t>((pieces * tiles + resident - 1) / resident, a.n_groups == 1 ? 8 : 16);
  // Of several matrices, whole sets of the tiles whose sums meet in LDS together, so that a workgroup's start is shared,
  // if every compute unit still has one (48 rows over 64 of 1280x1280 16.9 us without, 11.1 with; 32 over 128 of
  // 1024x2048 13.7, 12.3; 6 over 64 of 1280x1280 would be 7.4 instead of 6.2).
  if (a.n_groups > 1 && pieces * tiles >= kTogether * kComputeUnits) a.run = (a.run + kTogether - 1) / kTogether * kTogether;
  const dim3 grid((unsigned)(pieces * ((tiles + a.run - 1) / a.run)));
  auto go = [&](auto kernel, int together) {
    return launch_kernel(kernel, grid, dim3(64 * waves), (size_t)waves * MT * NT * together * 1024, stream, a);
  };
  if constexpr (MT == 1 && NT == 1 && U == 1)
    if (a.cin < kChunk) return go(k_matvec<X, 1, 1, 1, 1, 1, true, false, 1>, 1);
  if constexpr (MT == 1 && (X != kXF32 || U / P == 1))
    if (steps == 1)
      return a.run > 1 ? go(k_matvec<X, MT, NT, U, P, 2, true, true, kTogether>, kTogether) : go(k_matvec<X, MT, NT, U, P, 1, true, true, 1>, 1);
  // (of one row tile, only what launch_x sends more than one step of)
  if constexpr (MT > 1 || U == 4 || (X == kXF32 && (U == 1 || U / P > 1))) return go(k_matvec<X, MT, NT, U, P, 2, false, true, 1>, 1);
  return hipErrorInvalidValue;
}

// One group: the smallest piece that holds its rows.  Several: pieces of 4 rows where most groups have
// one or two (rows of popular groups then share a read of the weights only through the caches: 80 rows
// over 512 groups 35 us against 43, 320 rows 93 against 76) and for fp32 rows (320 rows 155 us against
// 205), otherwise of 16.
template <int X>
hipError_t launch_x(const Args& a, hipStream_t stream) {
  const int chunks = a.cin / kChunk;
  const bool one = a.n_groups == 1;
  const int64_t rows = one ? a.rows : (4 * a.rows <= a.n_groups || X == kXF32 ? 4 : 16);
  constexpr int kU = X == kXF32 ? 1 : 4;             // fp32 rows that fill the columns: 48 registers a chunk
  if (rows > 16 && chunks > 0) {
    // more channels at a time share the loads of x, as long as every compute unit has a workgroup
    const int tiles = (a.cout + 15) / 16;
    if (rows <= 32 || X == kXF32) {
      if (tiles > 512 && X != kXF32) return launch_tile<X, 2, X == kXF32 ? 2 : 3, 1, 1>(a, stream);
      return tiles > 256 ? launch_tile<X, 2, 2, 1, 1>(a, stream) : launch_tile<X, 2, 1, 1, 1>(a, stream);
    }
    if constexpr (X != kXF32) return tiles > 256 ? launch_tile<X, 4, 2, 1, 1>(a, stream) : launch_tile<X, 4, 1, 1, 1>(a, stream);
  }
  if (chunks <= 8) return launch_tile<X, 1, 1, 1, 1>(a, stream);
  if (chunks <= 16) return rows <= 8 ? launch_tile<X, 1, 1, 2, 2>(a, stream) : launch_tile<X, 1, 1, 2, 1>(a, stream);
  if (rows <= 4) return launch_tile<X, 1, 1, 4, 4>(a, stream);
  if (rows <= 8) return launch_tile<X, 1, 1, 4, 2>(a, stream);
  // 6 to 8 waves where 4 chunks a wave would leave fewer
  return chunks <= 24 ? launch_tile<X, 1, 1, X == kXF32 ? 1 : 3, 1>(a, stream) : launch_tile<X, 1, 1, kU, 1>(a, stream);
}

}  // namespace

hipError_t launch_matvec(const void* x, int x_type, const float* x_scale, int64_t x_scales, int64_t rows, int64_t cin,
                         int64_t cout, const int64_t* offsets, int64_t n_groups, const uint8_t* code, const uint8_t* fp4,
                         const float* amax, float gdiv, void* y, hipStream_t stream) {
  Args a{};
  a.x = x;
  a.x_scale = x_scale;
  a.code = code;
  a.fp4 = fp4;
  a.amax = amax;
  a.offsets = offsets;
  a.y = y;
  a.rows = rows;
  a.n_groups = n_groups;
  a.cout = (int)cout;
  a.cin = (int)cin;
  a.x_scales = (int)x_scales;
  a.gdiv = gdiv;
  if (x_type == kXBf16) return launch_x<kXBf16>(a, stream);
  return x_type == kXF32 ? launch_x<kXF32>(a, stream) : launch_x<kXE4m3>(a, stream);
}

}  // namespace lh

// Argument blocks and host-side planning of the selective scan, the short
// causal convolution and the norm around a block (pdssm_selscan_*,
// pdssm_conv_*, pdssm_norm_*): shared by the C ABI (host only) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "pdscan_linattn_plan.h"

namespace pdscan {

constexpr int kSsMaxN = 64;      // state values of a channel
constexpr int kSsMaxD = 1 << 20; // channels
constexpr int kCvMinW = 2, kCvMaxW = 4;

// The sequences of a call, cut into segments where there are few.
struct SsSegs {
  const int32_t* cu;             // packed: B+1 row offsets, NULL: B sequences of L steps
  const int32_t* table;          // packed and split: {sequence, first row, rows, first | last << 1} per segment
  int B, L, nseg, seg, segs;     // nseg per sequence (not packed), steps per segment, segments in all (bound)
};

// Indexes of pieces and tiles, also on the host.  Offsets of packed sequences
// that are out of order can ask for more pieces than there is room for; the
// table drops those behind the bound, and a run that names one gets the last.
constexpr int ss_piece_at(int first, int more, int pieces) {
  return first > pieces - 1 - more ? pieces - 1 : first + more;
}
// The gradient's tile at step t of piece `at` of sequence b, which starts at
// row t0: tiles of different pieces do not meet (per: tiles of a sequence, 0 where packed).
constexpr int64_t ss_tile_of(int per, int b, int at, int t0, int t, int tile) {
  return (per ? (int64_t)b * per : (int64_t)at) + t0 / tile + t / tile;
}

// Workgroups go to the eight dies in turn; this numbers them so that a die
// has neighbours: they share rows' cache lines and, in a scan, B and C.  At or
// past n: nothing to do; so is what the last of several rows of a grid has behind
// the eight dies' units, which would be the next die's first ones.
constexpr long long ss_near(unsigned id, long long n) {
  const long long per = (n + 7) / 8, at = id / 8;
  return at < per ? (long long)(id % 8) * per + at : n;
}

// One pass of the selective scan.  Element (b, t, d) of x, dt, z, y and their
// gradients is at sb b + st t + d; B and C have a head axis of G groups.
struct SsArgs {
  LaView x, dt, z, Bm, Cm, y;    // z.p NULL: no gate
  LaView gy, gx, gdt, gz;        // (gradient) gz.p NULL with z.p
  const float *A, *skip, *bias;  // [D][N]; [D] or NULL
  const float *h0, *ghL;         // [B][D][N] or NULL: zero
  float *hL, *gh0;               // gh0 may be NULL
  SsSegs s;                      // of this launch: pieces in the state pass, runs of `run` pieces in the others
  const int32_t *pieces, *runs;  // packed: first piece and first run of every sequence (runs NULL: whole sequences)
  int piece, npiece, run, npieces;   // steps of a piece, pieces of a sequence (not packed), of a run, in all
  float *seg, *adj;              // [pieces][D][N]: contributions of pieces, then entering (adjoint) states; NULL: one piece
  float *sum;                    // [pieces][D]: sums of the steps d_t of a piece
  float *ckpt, *cum;             // states at the tiles' starts, each piece from zero, and the sums up to there
  float *part;                   // partial g_B and g_C [2][blocks of all groups][rows][N]
  float* partA;                  // [segments][D N + 2 D]: g_A, g_skip, g_bias
  uint32_t* header;              // workspace header
  int D, N, G, softplus;
  unsigned row;                  // workgroups along x of the launch
  long long rows;                // token rows in all
};

struct SsCarryArgs {
  const float *A, *user[2];      // user: states before the first piece, adjoint states behind the last [B][D][N], NULL: zero
  float* seg[2];                 // of both directions; the second NULL: forwards only
  const float* sum;
  const int32_t* starts;         // packed: first piece of every sequence
  int B, D, N, npiece, blocks;
  unsigned row;
};

// Sums of `parts` rows of `width` columns, of which each output takes its share in turn (NULL: no more).
struct SsSumArgs {
  const float* part;
  float* out[3];
  int64_t share[3];
  float* mid;                    // [kSsSumMid][width] where there are more than kSsSumMost parts
  int parts;
  int64_t width;
};
// What finishes a scan's gradient: channel blocks' parts of g_B and g_C, and those sums.
struct SsFoldArgs {
  const float* part;
  LaView out[2];
  const int32_t* cu;
  int B, L, N, G, blocks;        // blocks per group
  long long rows;
  unsigned folds;                // workgroups of each of g_B and g_C; the sums' come behind them
  SsSumArgs sum;
};
constexpr int kSsSumMost = 256, kSsSumMid = 64;

struct SsStepArgs {
  LaView x, dt, z, Bm, Cm, y;
  const float *A, *skip, *bias;
  float* state;
  const int32_t* idx;
  int B, D, N, G, slots, softplus;
  unsigned row;
};

// States of a lane and lanes of a channel, by the state count: a wave holds
// 64 / lanes channels whole.
struct SsShape {
  int S, NS;
};
inline constexpr SsShape ss_shape(int N) {
  return N <= 8 ? SsShape{2, 4} : N <= 16 ? SsShape{4, 4} : N <= 32 ? SsShape{4, 8} : SsShape{8, 8};
}
inline constexpr int ss_channels(int N) { return 64 / ss_shape(N).NS; }   // of a wave
inline int ss_blocks(int K, int per) { return (K + per - 1) / per; }        // channel blocks of a group of K

// A tile is four waves of eight steps each.
constexpr int kSsFwdSteps = 8;
constexpr int kSsBwdSteps = 8, kSsTimeWaves = 4, kSsBwdTile = kSsBwdSteps * kSsTimeWaves;
constexpr int kSsBwdGroups = 1;   // channel groups of a gradient's workgroup: two would halve the partial g_B and g_C and were slower
constexpr int kSsStateGroups = 4;

// How a call cuts the step axis.  A piece is what a wave of the state pass
// takes; a run of pieces is what a workgroup of the others takes.
struct SsSplit {
  int piece, npiece, pieces;     // steps, of a sequence (not packed), in all (bound)
  int run, seg, nseg, segs;      // pieces of a run, its steps, runs of a sequence, in all (bound)
  bool cut;                      // sequences take more than one run
  bool states;                   // and more than one piece
};

// Time of `fill` times the workgroups that the card holds, `per` a compute unit,
// in rounds of it full: with one of three it is not three times as fast, but takes .6 of the time.
inline double ss_rounds(double fill, int per, bool bwd) {
  const double whole = (double)(long long)fill;
  const int left = (int)((fill - whole) * per + 0.999);
  if (left <= 0) return whole;
  if (left >= per) return whole + 1;
  return whole + (per == 3 ? (left == 1 ? (bwd ? 0.6 : 0.67) : (bwd ? 0.78 : 0.8)) : bwd ? 0.75 : 0.8);
}

// `width` workgroups take a run, `per` of them are on a compute unit at once;
// `states` workgroups take a piece of the state pass, a few of them a compute unit.
//
// A sequence that is not cut takes its steps one after another: its time goes
// by rounds of the card.  Cut, time goes by the work, 1.45 times it
// forwards and 1.08 backwards (the state passes), and the launches add what 280 and 100
// steps take.  768 channels of 16 states (16 sequences fill the card once), bf16, in us, uncut / cut:
//   forwards   512 steps of 1: 28 / 27, of 4: 30 / 33;  1024 of 1: 50 / 28, of 4: 53 / 46;  2048 of 6: 117 / 101, of 8: 114 / 116, of 12: 142 / 163
//   backwards  256 of 1: 61 / 50;  384 of 4: 81 / 64;  2048 of 8: 389 / 311, of 12: 499 / 449, of 16: 529 / 567, of 20: 727 / 700, of 24: 848 / 842
// Sequences of different lengths, where the longest counts, are taken as three of a third of the rows:
//   16 in 2048 rows 33 / 45 and 111 / 94, 16 in 8192 102 / 89 and 333 / 215; 2048 channels, 40 in 8192 191 / 242 and 713 / 716
// That suits lengths with a long tail, as drawn for these.  Where all are alike it cuts what would fill the card
// whole (the same sequences in a batch / packed): forwards 40 of 512 94 / 170, 16 of 2048 141 / 231, 32 of 2048 253 / 487;
// backwards 348 / 472, 536 / 679, 1037 / 1514.  Whoever has such lengths is better off with a batch.
inline SsSplit ss_split(int B, int L, int packed, long long width, int per, long long states, bool bwd) {
  SsSplit s;
  constexpr int kCus = 256, kUnit = 32, kLeast = 64, kRun = 128;   // steps of a piece and of a run, at least
  const long long seqs = packed ? 1 : B, room = (long long)per * kCus;
  const int like = packed ? (B < 3 ? B : 3) : B;
  const double fill = (double)like * width / room, steps = (double)L / (packed ? like : 1);
  const bool pays = (bwd ? 1.08 : 1.45) * fill + (bwd ? 100.0 : 280.0) / steps < ss_rounds(fill, per, bwd);
  // Runs cost the state passes, not their number: where sequences are cut, four times the room evens out the end.
  long long n = pays ? (4 * room + seqs * width - 1) / (seqs * width) : 1;
  if (n > L / kRun) n = L / kRun;
  s.cut = n > 1;
  long long m = (s.cut || bwd) ? (4 * 256 + seqs * states - 1) / (seqs * states) : 1;   // pieces
  if (m > L / kLeast) m = L / kLeast;
  if (m < n) m = n;
  if (m < 1) m = 1;
  s.run = s.cut ? (int)((m + n - 1) / n) : 0x7fffffff;
  if (s.cut) m = n * s.run;
  s.piece = m > 1 ? (int)(((L + m - 1) / m + kUnit - 1) / kUnit * kUnit) : L;
  s.npiece = (int)(((long long)L + s.piece - 1) / s.piece);
  s.states = s.npiece > 1;
  if (!s.states) s.cut = false;
  s.seg = s.cut ? s.piece * s.run : L;
  s.nseg = s.cut ? (int)(((long long)L + s.seg - 1) / s.seg) : 1;
  auto all = [&](int len, int each, bool more) {
    const long long k = !packed ? (long long)B * each : more ? (long long)(L / len) + B : B;
    return k > 0x7fffffffll ? 0x7fffffff : (int)k;
  };
  s.pieces = all(s.piece, s.npiece, s.states);
  s.segs = all(s.seg, s.nseg, s.cut);
  return s;
}

struct CvArgs {
  LaView x, y, gy, gx;
  const float *w, *bias;         // [D][W]; [D] or NULL
  const void *x0, *gxL;          // [B][W-1][D] or NULL: zero
  void *xL, *gx0;                // gx0 may be NULL
  const int32_t* cu;
  float* part;                   // [parts][D][W], [D]
  uint32_t* header;              // workspace header
  int B, L, D, W, silu, strips;  // strips: of a sequence (packed: of all rows)
  int parts;
  unsigned units;                // threads with rows to do, before those of the states
  unsigned row;
};
struct CvStepArgs {
  LaView x, y;
  const float *w, *bias;
  void* state;                   // [slots][W-1][D]
  const int32_t* idx;
  int B, D, W, silu, slots;
  unsigned row;
};
constexpr int kCvRows = 16;      // rows of a thread, forwards
inline long long cv_units(const CvArgs& a, int bf16) {
  return (long long)(a.cu ? 1 : a.B) * ((a.L + kCvRows - 1) / kCvRows) * (a.D / (bf16 ? 8 : 4));
}
constexpr int kCvBwdRows = 32;   // backwards
constexpr int kCvBwdStrips = 4;  // strips of a workgroup, backwards

// Lanes of a row and 16-byte vectors of a lane, by the row's length.
struct NmShape {
  int P, K;                      // P: 1 .. 64, or 256 (a whole workgroup)
};
inline constexpr NmShape nm_shape(int d, int bf16) {
  const int n = d / (bf16 ? 8 : 4);
  if (n > 256) return NmShape{256, n <= 512 ? 2 : n <= 1024 ? 4 : 8};
  if (n > 64) return NmShape{64, n <= 128 ? 2 : 4};
  int p = 1;
  while (p < n) p *= 2;
  return NmShape{p, 1};
}
constexpr int kNmMaxD = 8192;

struct NmArgs {
  LaView x, z, r, y;             // [B][H][L][d]; z.p, r.p may be NULL
  LaView gy, gx, gz;
  const float *w, *s;            // [H][d] or [d]; s may be NULL
  float* part;                   // (gradient) sums of a workgroup's rows, for w and behind them for s
  int64_t part_chunk, part_head, part_s;   // floats between those of chunks, heads, and the two
  uint32_t* header;              // workspace header
  int B, H, L, d, gate, per_head;
  int cols, slots, tiles;        // lanes of a workgroup side by side in (head, row), rows at once, tiles of the former
  int chunks;                    // workgroups along the rows
  float eps;
  long long rows;                // B L: of a head
  unsigned row;
};
// Heads side by side where they lie so (`near`: the head stride is below the step's), else one head a workgroup.
inline void nm_plan(NmArgs& a, int bf16, bool near, int each, int most) {
  const int P = nm_shape(a.d, bf16).P;
  const long long all = (long long)a.H * P;
  a.cols = !near ? P : all < 256 ? (int)all : 256;
  a.slots = 256 / a.cols;
  a.tiles = (int)((all + a.cols - 1) / a.cols);
  long long n = (a.rows + (long long)a.slots * each - 1) / ((long long)a.slots * each);
  if (most && n > most) n = most;
  a.chunks = (int)(n > 0x7fffffff ? 0x7fffffff : n);
}

}  // namespace pdscan

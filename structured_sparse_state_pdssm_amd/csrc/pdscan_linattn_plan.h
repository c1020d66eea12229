// Argument blocks and host-side planning of the linear-attention passes
// (pdssm_linattn_*): shared by the C ABI (host only) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

namespace pdscan {

constexpr int kLaChunk = 64;     // segments are multiples of this: one or two chunks
constexpr int kLaMaxD = 256;     // widest key or value row
constexpr int kLaMaxStep = 1 << 23;   // longest step stride, elements: 64 rows stay within 31 bits of bytes
constexpr int kLaPiece = 512;    // longest segment of a gradient (see the log-decay gradient)
constexpr double kLaNear = 24.0; // log2 of the decay over a chunk up to which it is split into factors of its tokens
constexpr int kLaHeader = 256;   // workspace header: word 1 stays zero (nothing here waits on another workgroup)

enum { kLaFwd, kLaQ, kLaK, kLaV };   // jobs of the product kernel

// A strided tensor: element strides of the batch, head and step axes; the
// last axis is contiguous.
struct LaView {
  void* p;
  int64_t sb, sh, st;
};

// One product o = form(x, y, z) over every sequence (see pdscan_linattn.h).
struct LaJob {
  LaView x, y, z, o, w;
  int xd, yd, zd, od, wd;      // heads of the pass per head of the view
  int DK, DV;                  // widths of x, y rows and of z, o rows
  const float* s_user;         // state before the first step in the job's direction [B][H], NULL: zero
  const float* s_seg;          // entering states of the other segments [segment][H]
  float* s_fin;                // state after the last step [B][H], NULL: not written
  const float* xd_with;        // state to dot the final state with [B][H], NULL: none
  double* xd_out;              // that product [slab][segment][H]
  float* seg_out;              // (state pass) contributions [segment][H], written at the next segment
  float* seg_decay;            // (state pass) the segment's decay [segment][H]
  float* dot;                  // w . o per token [slab][H][rows], NULL: none
  int sm, sn;                  // strides of a state's x-row and z-row axes
  float s_out, s_ratio, s_upd; // scale of the output, of its own tokens' part beside the state's, of the update
  int mode;                    // kLaFwd ..
  int rev;                     // 1: backwards in time (kLaK and kLaV)
  int o_f32;                   // 1: o is fp32 whatever the inputs' type
};

struct LaArgs {
  LaView g;                    // log decay, fp32
  const int32_t* cu;           // packed: B+1 row offsets, NULL: B sequences of L steps
  const int32_t* table;        // packed and split: {sequence, first row, rows, first | last << 1} per segment
  uint32_t* header;            // workspace header
  int B, H, L, nseg, seg, segs;   // nseg per sequence (not packed), steps per segment, segments in all (bound)
  int slabs, njobs;
  unsigned row;                // workgroups along x of the launch
  long long rows, state;       // token rows in all; elements of one state
  LaJob job[3];
};

struct LaStepArgs {
  LaView q, k, v, g, o;
  float* state;
  const int32_t* idx;
  int B, H, qd, dk, dv, slots, cols;   // cols: value columns per workgroup
  unsigned row;                // workgroups along x of the launch
  float scale;
  int bf16;
};

// Finishing pass of the gradient: log-decay gradient of one segment and head.
struct LaDecayArgs {
  LaArgs c;
  const float* r;              // q . dq per token [slabs][H][rows]
  const float* k;              // k . dk per token [slabs][H][rows]
  const float* sS;             // entering states [segment][H]
  const float* sR;             // entering adjoints [segment][H]
  const double* xd;            // final state . its gradient [slabs][segment][H], NULL: zero
  double* part;                // sums per segment and head (one decay per head)
  LaView out;
  const float *h0, *g_h0;      // states before the sequences and their gradients [B][H], NULL: zero, not asked for
  int slabs, per_head;
};

// Sum over the value heads that share a query or key head.
struct LaFoldArgs {
  const float *part_q, *part_k;   // [rows][H][d]
  LaView out_q, out_k;
  const int32_t* cu;
  int B, H, L, ratio, d, bf16;
  long long rows;
};

inline constexpr int la_pad(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Waves of a workgroup, 32 columns each, for x rows of DK and z rows of DV
// elements.  Rows of more than 128 elements take more waves than columns need
// where fewer would not hold the tiles under way in their registers.
inline constexpr int la_waves(int DK, int DV, int bf16) {
  const int w = DV <= 32 ? 1 : DV <= 64 ? 2 : 4;
  return DK <= 128 ? w : bf16 ? (w < 2 ? 2 : w) : 4;
}
inline constexpr int la_slabs(int DK, int DV, int bf16) {
  const int w = 32 * la_waves(DK, DV, bf16);
  return (DV + w - 1) / w;
}
// Passes of the product and state kernels.
enum { kLaPassState, kLaPassFwd, kLaPassQK, kLaPassV, kLaPassQKV };
// Whether the three jobs of a gradient have one shape and go in one launch.
inline constexpr bool la_one(int dk, int dv, int bf16) {
  return la_pad(dk) == la_pad(dv) && la_slabs(dv, dk, bf16) == la_slabs(dk, dv, bf16) &&
         la_waves(dk, dv, bf16) == la_waves(dv, dk, bf16);
}
// Whether any dk and dv take a pass to the kernel of x rows of up to `pad`
// elements and `waves` waves.
inline constexpr bool la_reached(int pass, int pad, int waves, int bf16) {
  for (int dk = 8; dk <= kLaMaxD; dk += 8)
    for (int dv = 8; dv <= kLaMaxD; dv += 8) {
      const bool one = la_one(dk, dv, bf16);
      if ((pass == kLaPassQKV && !one) || ((pass == kLaPassQK || pass == kLaPassV) && one)) continue;
      const bool q = pass == kLaPassQK || pass == kLaPassQKV;   // x rows of dv, z rows of dk
      if (la_pad(q ? dv : dk) == pad && la_waves(q ? dv : dk, q ? dk : dv, bf16) == waves) return true;
    }
  return false;
}
// Registers of a lane that the state and the outputs (`tiles` of 32 x 32 a
// wave) and the tiles under way (`units` of 16 bytes a lane) take; an fp32 unit
// counts its pieces on their way to LDS too.
inline constexpr int la_regs(int tiles, int units, bool f32) { return 16 * tiles + (f32 ? 11 * units / 2 : 4 * units); }
// Waves of a product kernel on a SIMD: two, and one where two spill more than
// the second hides.  One count for all jobs of a width, by the forward pass: 65536 steps
// of 128/128 bf16 (144 registers) 262 us with two, 369 with one; 8 x 2048 steps,
// 12 heads in fp32: 128/128 (146) 239 and 291 forwards, where two spill nothing,
// and 667 and 762 for the gradient, whose jobs spill 8 to 44; the gradient of
// 32/64 (158) 245 and 193; 2 x 2048 steps, 8 heads, 256/256 bf16 (216) 115 and 91.
// Three change nothing where they fit.
inline constexpr int la_simd_waves(int regs) { return regs <= 150 ? 2 : 1; }
// Tokens of a chunk.  64 where four waves share the scores (bf16); else 32, which
// halves the registers and the LDS of a workgroup (two waves a SIMD
// instead of one: 24 heads of 64/32 at 16 x 2048 tokens 122 -> 104 us).
inline constexpr int la_chunk(int waves, int bf16) { return waves < 4 || !bf16 ? 32 : 64; }
// Bytes of LDS that a workgroup of the product kernel takes with scores of
// `pieces` pieces (LaTile lays them out).
inline constexpr int la_lds(int pad, int waves, int bf16, int pieces) {
  const int C = la_chunk(waves, bf16);
  return C * (bf16 ? 2 : 6) * (2 * pad + 32 * waves) + (waves == 4 && bf16 ? pieces * C * C * 2 : 0) +
         4 * (64 / C * (8 * C + 8) + (waves + 1) * C);
}
// Workgroups of the product kernel that a compute unit holds, by LDS (160 KiB)
// and by those waves.
inline int la_resident(int DK, int DV, int bf16, int bwd) {
  const int es = bf16 ? 2 : 4, nw = la_waves(DK, DV, bf16), d = la_pad(DK), C = la_chunk(nw, bf16);
  const int lds = la_lds(d, nw, bf16, bwd ? 3 : 2);
  const int waves = 4 * la_simd_waves(la_regs((d + C) / 32, C * es * (2 * d + 32 * nw) / (1024 * nw), !bf16));
  const int n = 163840 / lds < waves / nw ? 163840 / lds : waves / nw;
  return n < 1 ? 1 : n;
}

struct LaSplit {
  int seg, nseg, segs;         // steps per segment, segments per sequence (not packed), bound in all
  bool split;
};

// Cuts the step axis into segments so that a launch of `width` workgroups per
// segment fills the card once (`room` workgroups).  Whole sequences where
// they do that, and up to 256 steps: the three launches more cost what the
// shorter chains save.  Sequences of different lengths take 7/4 of it, so that
// no long one is left alone at the end.  A segment's states are written and
// read twice; with at least a workgroup a compute unit they stay under half of
// what its steps (`bytes` each) move.  No segment is over `longest` steps.
//   65536 steps, 16 heads, 128/128 bf16: 2048 steps 405 us, 1024 449, 4096 423, uncut over 5000
//   16 x 2048 steps, 24 heads, 64/32 bf16: 448 steps 111 us (512 103, 256 119), uncut 125
//   4 x 4096 steps, 8 heads, 16/64 fp32: 128 steps 46 us, 64 62, 256 63
//   23 sequences in 12001 rows, 24 heads, 128/64 bf16: 384 steps 105 us, 192 117, 640 124
//   gradient of 9 in 8190 rows, 16 heads, 128/128 bf16: 512 steps 243 us, 384 254, 256 275
inline LaSplit la_split(int B, int L, int packed, long long width, int room, long long state, int bytes, int longest) {
  LaSplit s;
  long long n = (long long)room / (packed ? width : B * width);   // segments of a sequence
  if (packed) n = n * 7 / 4;
  const long long least = 256 / (packed ? width : B * width), most = (long long)L * bytes / (32 * state);
  if (n > most) n = most > least ? most : least < n ? least : n;
  if (n > (L - 1) / kLaChunk + 1) n = (L - 1) / kLaChunk + 1;
  if (n < ((long long)L + longest - 1) / longest) n = ((long long)L + longest - 1) / longest;
  s.split = n > 1 && L > 256;
  const long long each = s.split ? ((long long)L + n - 1) / n : L;
  s.seg = each <= 5 * kLaChunk / 4 && s.split ? kLaChunk : (int)((each + kLaChunk - 1) / kLaChunk * kLaChunk);
  s.nseg = s.split ? (int)(((long long)L + s.seg - 1) / s.seg) : 1;
  const long long segs = !packed ? (long long)B * s.nseg : s.split ? (long long)(L / s.seg) + B : B;
  s.segs = segs > 0x7fffffffll ? 0x7fffffff : (int)segs;
  return s;
}

// Workgroups that read the same rows (the jobs, slabs and heads of one segment
// and query / key head) follow one another, on eight dies in turn: the cache
// behind the dies serves them as fast as keeping each such set on one die and
// its L2 would (product kernels of 32 to 128 wide rows, 12 to 24 heads, shared
// or not: 179 us so against 189 and 178, 216 / 214, 70 / 70, 68 / 66).
inline long long la_grid(const LaArgs& a) { return (long long)a.segs * a.H * a.slabs * a.njobs; }

// A launch has fewer than 2^32 threads along an axis, which is 2^23 workgroups
// of 512: more take rows of equal length along y, in the same order.  Numbers
// at or behind `blocks` (fewer than y of them) have nothing to do.
struct LaGrid {
  unsigned x, y;
};
inline LaGrid la_grid_rows(long long blocks, int threads) {
  const long long most = 0xffffffffll / threads;
  const long long y = (blocks + most - 1) / most;
  return LaGrid{(unsigned)((blocks + y - 1) / y), (unsigned)y};
}

inline size_t la_align(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace pdscan

// Argument blocks and host-side planning of the linear-attention passes
// (pdssm_linattn_*): shared by the C ABI (host only) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

namespace pdscan {

constexpr int kLaChunk = 64;     // tokens per step of a sequence's serial axis (32 for wide fp32 rows)
constexpr int kLaMaxD = 256;     // widest key or value row
constexpr int kLaMaxStep = 1 << 23;   // longest step stride, elements: 64 rows stay within 31 bits of bytes
constexpr int kLaKeep = 512;     // steps of a segment between states kept for the log-decay gradient
constexpr int kLaHeader = 256;   // workspace header: word 1 stays zero (nothing here waits on another workgroup)

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
  float* seg_decay;            // (state pass) log2 decay of the segment [segment][H]
  float* keep;                 // states inside a segment, every kLaKeep steps [row / kLaKeep][H], NULL: none
  float* dot;                  // w . o per token [slab][H][rows], NULL: none
  int sm, sn;                  // strides of a state's x-row and z-row axes
  float s_inter, s_intra, s_upd;
  int rev;                     // 1: backwards in time
  int o_f32;                   // 1: o is fp32 whatever the inputs' type
};

struct LaArgs {
  LaView g;                    // log decay, fp32
  const int32_t* cu;           // packed: B+1 row offsets, NULL: B sequences of L steps
  const int32_t* table;        // packed and split: {sequence, first row, rows, first | last << 1} per segment
  uint32_t* header;            // workspace header
  int B, H, L, nseg, seg, segs;   // nseg per sequence (not packed), steps per segment, segments in all (bound)
  int slabs, njobs;
  long long rows, state;       // token rows in all; elements of one state
  LaJob job[3];
};

struct LaStepArgs {
  LaView q, k, v, g, o;
  float* state;
  const int32_t* idx;
  int B, H, qd, dk, dv, slots, cols;   // cols: value columns per workgroup
  float scale;
  int bf16;
};

// Finishing pass of the gradient: log-decay gradient of one segment and head.
struct LaDecayArgs {
  LaArgs c;
  const float* r;              // q . dq per token [r_slabs][H][rows]
  const float* k;              // k . dk per token [k_slabs][H][rows]
  const float* sS;             // entering states [segment][H]
  const float* sR;             // entering adjoints [segment][H]
  const float* kS;             // the same every kLaKeep steps inside a segment [row / kLaKeep][H]
  const float* kR;
  const double* xd;            // final state . its gradient [xd_slabs][segment][H], NULL: zero
  double* part;                // sums per piece of kLaKeep steps and head (one decay per head)
  LaView out;
  int r_slabs, k_slabs, xd_slabs, per_head;
  int subs;                    // pieces of kLaKeep steps of the longest segment
};

// Sum over the value heads that share a query or key head.
struct LaFoldArgs {
  const float* part;           // [rows][H][d]
  LaView out;
  const int32_t* cu;
  int B, H, L, ratio, d, bf16;
  long long rows;
};

inline int la_pad(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 128 ? 128 : 256; }
inline int la_waves(int d) { return d <= 32 ? 1 : d <= 64 ? 2 : 4; }          // 32 columns each
inline int la_slabs(int d) { return (d + 32 * la_waves(d) - 1) / (32 * la_waves(d)); }

struct LaSplit {
  int seg, nseg, segs;         // steps per segment, segments per sequence (not packed), bound in all
  bool split;
};

// Steps per segment of a pass with `width` workgroups per segment.
inline LaSplit la_split(int B, int L, int packed, int width) {
  LaSplit s;
  const long long rows = packed ? (long long)L : (long long)B * L;
  const long long want = 1024;
  long long seg = (rows * width + want - 1) / want;
  if (seg < 256) seg = 256;
  seg = (seg + kLaChunk - 1) / kLaChunk * kLaChunk;
  if (seg >= L || (!packed && (long long)B * width >= want / 2)) {
    s.seg = (int)((L + (long long)kLaChunk - 1) / kLaChunk * kLaChunk > 0x7fffffc0ll ? 0x7fffffc0ll
                  : (L + (long long)kLaChunk - 1) / kLaChunk * kLaChunk);
    s.nseg = 1;
    s.segs = B;
    s.split = false;
    return s;
  }
  s.seg = (int)seg;
  s.nseg = (int)((L + seg - 1) / seg);
  const long long n = packed ? (long long)(L / seg) + B : (long long)B * s.nseg;
  s.segs = n > 0x7fffffffll ? 0x7fffffff : (int)n;
  s.split = true;
  return s;
}

inline int la_subs(const LaSplit& s, int L) { return ((s.seg < L ? s.seg : L) + kLaKeep - 1) / kLaKeep; }

inline size_t la_align(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace pdscan

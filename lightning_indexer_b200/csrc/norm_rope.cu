// RMS norm of query and key heads and the position rotation in one pass over the rows, its
// gradients, and the same pass writing new keys and values into a paged cache (sm_100a).
//
// A row is one head of one token, x[0..D).  With weight g (or none: n = x):
//   n = x * rstd * g,  rstd = 1 / sqrt(mean(x^2) + eps)
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a),  a = position * inv_freq[i],
// on the pairs (n_i, n_{i+r/2}) or, interleaved, (n_2i, n_{2i+1}), i < r/2; dims past r pass.
// Gradient, from dy: dn = the pair rotation by -a of dy, then with xh = x * rstd
//   dg = sum over rows of dn * xh,   dx = rstd * (dn * g - xh * mean(dn * g * xh)).
// Everything is fp32 from the bf16 inputs to the one rounding of each output.
//
// The angle's fraction of a turn is an integer product (see turn_step): at position 10^6 an
// fp32 product would be off by 0.06 rad, this one by 1e-7 rad.  cos and sin are computed once
// per token and warp and reused over the token's heads.
//
// Layout: D / 16 lanes hold one row, 16 elements each in two 16-byte pieces chosen so that
// both members of a rotation pair sit in the same lane, so the only exchange between lanes
// is the norm's sum (and, backward, its dot product).  A warp takes 512 / D rows at once, a
// group, and runs over consecutive groups: their rows stream through a private ring in shared
// memory by asynchronous copies (no registers held while they fly), and the places of the
// run's tokens (sequence, position, page) are looked up by its lanes side by side, one chain
// of dependent loads per run instead of one per group.
//
// Bound by HBM (4 bytes an element forward, 6 backward), with about 210 instructions a group of
// 1 KiB forward, 300 backward (63 and 58 % of the issue slots).  Measured: 32768 tokens of
// 32 + 4 heads of 128 in 95 to 103 us (6.3 to 5.9 TB/s), the backward of 65536 in 303 to 320 us
// (6.0 to 5.7 TB/s; 128 registers a thread, of which the <128, 0> form spills 28 bytes), an append
// of 32768 tokens (4 + 4 heads and the indexer's key) in 30 us (5.0 TB/s: every group of K is
// another token, whose turns it computes for itself; its 2304 blocks are 3.1 waves).  The form for
// tensors that do not agree in width or pairing spills 68 bytes: the same append takes 30.3 us
// with interleaved pairs where it takes 29.2 without, and 22.6 at d = 64 with d_I = 128 (floor 12.8).
#include <algorithm>

#include "common.cuh"

namespace dsa {

// One tensor of rows: token t's heads are `heads` consecutive rows of D elements.
struct HeadSeg {
  const uint16_t* x;    // [T, heads, D], token stride x_stride (elements)
  const uint16_t* dy;   // backward only: gradient at the output, token stride dy_stride
  uint16_t* y;          // output rows (forward), gradient rows (backward)
  int x_stride, dy_stride;  // elements from token to token
  long long y_stride;       // the same of the output, or of a page when paged
  const uint16_t* g;    // [D] or null: no norm
  const double* inv_freq;  // [rotary / 2] or null
  int heads, D, rotary;
  int interleaved, paged;
  int block0;           // first block of this tensor's rows
  int groups;           // warp-sized groups of 512 / D rows
  int iters;            // groups of a run, at most 32 tokens' worth
  int warps;            // warps of this tensor (whole blocks)
  unsigned div_mul;     // row / heads = (row * div_mul) >> div_shift for rows < 2^31
  int div_shift;
  float* dg_part;       // backward with norm: [blocks of this tensor][D]
};

// Where a token belongs.  Sequence b owns the tokens cu[b] .. cu[b+1]; its last new token
// sits at position lens[b] - 1 (lens null: its first one at position 0).  Without offsets,
// token t is the one new token of sequence t (lens given) or at position t of one sequence.
struct TokenMap {
  const int* positions;  // [T] or null: rotation positions
  const int* cu;         // [batch + 1] or null
  const int* lens;       // [batch] or null
  int batch;
  int T;
  const int* table;  // [batch, table_width] page ids (paged outputs)
  int table_width, page_shift, num_pages;
};

constexpr int NR_MAX_SEGS = 5;
constexpr int NR_FWD_WARPS = 4;  // warps of a block; 5 blocks per SM: at most 102 registers (8 x 3 spills, 8 x 2 waits)
constexpr int NR_BWD_WARPS = 8;  // 2 blocks per SM
constexpr int NR_BWD_BLOCKS = 2 * 148;

struct HeadRowsParams {
  HeadSeg seg[NR_MAX_SEGS];
  int nseg;
  int zero_outside;  // rows of tokens outside the sequences (offsets given): 0 stay as they are, 1 become zeros
  int zero_block0;   // forward: the first of the blocks that write those zeros
  float eps;
  TokenMap tk;
};

// The token's sequence, or -1 past the last one.  Equal lengths are found at the first look.
__device__ __forceinline__ int token_seq(const TokenMap& tk, int t) {
  const int b0 = (int)((long long)t * tk.batch / tk.T);
  if (tk.cu[b0] <= t && t < tk.cu[b0 + 1]) return b0;
  if (t < tk.cu[0] || t >= tk.cu[tk.batch]) return -1;
  int lo = 0, hi = tk.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tk.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Rotation position of token t and, for a paged output, the element offset of its rows;
// false where the token writes nothing (past the last sequence, no page).
__device__ __forceinline__ bool place_token(const TokenMap& tk, const HeadSeg& s, int t, int& pos, long long& yoff) {
  pos = t;
  yoff = (long long)t * s.y_stride;
  if (t >= tk.T) return false;
  int b = 0;
  if (tk.cu) {
    b = token_seq(tk, t);
    if (b < 0) return false;
    pos = t - tk.cu[b] + (tk.lens ? tk.lens[b] - (tk.cu[b + 1] - tk.cu[b]) : 0);
  } else if (tk.lens) {
    b = t;
    pos = tk.lens[t] - 1;
  }
  if (s.paged) {
    const int pg = pos >> tk.page_shift;
    if (pos < 0 || pg >= tk.table_width) return false;
    const int page = tk.table[(long long)b * tk.table_width + pg];
    if ((unsigned)page >= (unsigned)tk.num_pages) return false;
    yoff = page * s.y_stride + (long long)(pos & ((1 << tk.page_shift) - 1)) * s.heads * s.D;
  }
  if (tk.positions) pos = tk.positions[t];
  return true;
}

// Turns per position as a 64-bit binary fraction: position * step, taken modulo 2^64 by the
// integer product itself, is the angle's fraction of a turn, exact however far the position.
__device__ __forceinline__ unsigned long long turn_step(double inv_freq) {
  double y = inv_freq * 0.15915494309189533577;  // radians to turns
  y -= floor(y);
  return __double2ull_rn(y * 18446744073709551616.0);
}

// cos and sin of an angle given in 2^-32 turns: the nearest quarter turn is taken off, the
// rest, at most pi / 4 either way, goes through the Taylor polynomials of both (remainders
// z^11 / 11! and z^10 / 10!: below 3e-8).
__device__ __forceinline__ void turn(uint32_t angle, float& c, float& s) {
  const uint32_t q = (angle + 0x20000000u) >> 30;
  const float z = (float)(int)(angle - (q << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z2 = z * z;
  float ps = fmaf(z2, 2.7557319e-6f, -1.9841270e-4f);
  ps = fmaf(ps, z2, 8.3333333e-3f);
  ps = fmaf(ps, z2, -1.6666667e-1f);
  const float sz = fmaf(ps * z2, z, z);
  float pc = fmaf(z2, 2.4801587e-5f, -1.3888889e-3f);
  pc = fmaf(pc, z2, 4.1666667e-2f);
  pc = fmaf(pc, z2, -0.5f);
  const float cz = fmaf(pc, z2, 1.f);
  const bool odd = q & 1u;
  s = __uint_as_float(__float_as_uint(odd ? cz : sz) ^ ((q & 2u) << 30));
  c = __uint_as_float(__float_as_uint(odd ? sz : cz) ^ (((q + 1u) & 2u) << 30));
}
__device__ __forceinline__ uint32_t angle_at(unsigned long long step, int pos) {
  return (uint32_t)(((unsigned long long)(long long)pos * step) >> 32);
}

// Two fp32 values in one 64-bit register pair: one instruction does both products, which
// counts here because the issue slots, not the memory, are what these kernels run out of.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// eight bf16 <-> four pairs
__device__ __forceinline__ void unpack8(const uint4& v, F2* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const F2* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = f2_get(f[i]);
    const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane holds of every row of its segment: two 8-element pieces at e0 and e1, each
// instruction of the row's lanes covering whole 16-byte pieces side by side.
template <int D, bool INTER>
struct LaneCols {
  static constexpr int LPR = D / 16;       // lanes per row
  static constexpr int RPW = 32 / LPR;     // rows per warp
  int sub;
  int e0, e1;
  bool rot0, rot1;  // whether the pairs 0-3 and 4-7 of this lane rotate

  __device__ __forceinline__ LaneCols(const HeadSeg& s, int sub_) : sub(sub_) {
    const int r16 = s.inv_freq ? s.rotary / 16 : 0;
    if (INTER) {  // pairs lie inside a piece
      e0 = 8 * sub;
      e1 = e0 + D / 2;
      rot0 = e0 < 16 * r16;
      rot1 = e1 < 16 * r16;
    } else {  // pair p is element p of the two pieces; the lanes past r16 share the dims that pass
      rot0 = rot1 = sub < r16;
      e0 = rot0 ? 8 * sub : 8 * (sub + r16);
      e1 = rot0 ? 8 * (sub + r16) : 8 * (sub + LPR);
    }
  }
  __device__ __forceinline__ bool rotates(int p) const { return p < 4 ? rot0 : rot1; }
  __device__ __forceinline__ int freq(int p) const {
    return INTER ? (p < 4 ? 4 * sub + p : 4 * sub + D / 4 + p - 4) : 8 * sub + p;
  }
};

// The turn steps of the block's segment and, per warp, the (cos, sin) of one token's pairs.
struct TurnSmem {
  unsigned long long step[64];
  __align__(16) float2 cs[NR_BWD_WARPS][64];
};
static_assert(NR_FWD_WARPS <= NR_BWD_WARPS, "one exchange buffer per warp");
__device__ __forceinline__ void load_steps(const HeadSeg& s, TurnSmem& ts) {
  if (!s.inv_freq) return;  // block-uniform
  if (threadIdx.x < s.rotary / 2) ts.step[threadIdx.x] = turn_step(s.inv_freq[threadIdx.x]);
  __syncthreads();
}

// cos and sin of this lane's eight rotation pairs, two by two.
struct LaneTurns {
  F2 c[4], s[4];
};

// Where the turn of frequency f lies in the exchange buffer: two to a 16-byte piece, the pieces
// that a row's lanes read together side by side.
__device__ __forceinline__ int cs_slot(int f) { return (((f >> 1) & 3) * 8 + (f >> 3)) * 2 + (f & 1); }

// This lane's turns at its row's position.  Where every row of the warp belongs to one token,
// the lanes compute the token's rotary / 2 pairs side by side and exchange them through
// shared memory.
template <bool SHARED, bool FULL, int D, bool INTER>
__device__ __forceinline__ void lane_turns(const HeadSeg& s, const LaneCols<D, INTER>& col, TurnSmem& ts, int pos,
                                           LaneTurns& L) {
  const int lane = threadIdx.x % 32;
  if (SHARED) {
    float2* cs = ts.cs[threadIdx.x / 32];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < (D + 63) / 64; ++j)
      if (const int f = 32 * j + lane; f < s.rotary / 2) turn(angle_at(ts.step[f], pos), cs[cs_slot(f)].x, cs[cs_slot(f)].y);
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; p += 2) {
      const float4 v = FULL || col.rotates(p) ? *reinterpret_cast<const float4*>(cs + cs_slot(col.freq(p))) : make_float4(1.f, 0.f, 1.f, 0.f);
      L.c[p / 2] = f2(v.x, v.z);
      L.s[p / 2] = f2(v.y, v.w);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; p += 2) {
      float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;
      if (col.rotates(p)) {
        turn(angle_at(ts.step[col.freq(p)], pos), c0, s0);
        turn(angle_at(ts.step[col.freq(p) + 1], pos), c1, s1);
      }
      L.c[p / 2] = f2(c0, c1);
      L.s[p / 2] = f2(s0, s1);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Pair rotation of the lane's 16 values (two pieces) by the turns' angles, or back by them.
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate16(F2* a, F2* b, bool rot0, bool rot1, const LaneTurns& L) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (!(half ? rot1 : rot0)) continue;  // dims that pass stay out of every product
#pragma unroll
    for (int i = 2 * half; i < 2 * half + 2; ++i) {
      if (INTER) {  // pairs 2 i and 2 i + 1: the words 2 (i & 1) and 2 (i & 1) + 1 of this half's piece
        const float2 c = f2_get(L.c[i]), sn = f2_get(L.s[i]), s = BACK ? make_float2(-sn.x, -sn.y) : sn;
        F2* x = (half ? b : a) + 2 * (i & 1);
        const float2 x0 = f2_get(x[0]), x1 = f2_get(x[1]);
        x[0] = f2(fmaf(x0.x, c.x, -(x0.y * s.x)), fmaf(x0.y, c.x, x0.x * s.x));
        x[1] = f2(fmaf(x1.x, c.y, -(x1.y * s.y)), fmaf(x1.y, c.y, x1.x * s.y));
      } else {
        const F2 u = a[i], v = b[i];
        a[i] = BACK ? fma2(u, L.c[i], mul2(v, L.s[i])) : sub2(mul2(u, L.c[i]), mul2(v, L.s[i]));
        b[i] = BACK ? sub2(mul2(v, L.c[i]), mul2(u, L.s[i])) : fma2(v, L.c[i], mul2(u, L.s[i]));
      }
    }
  }
}

__device__ __forceinline__ int row_token(const HeadSeg& s, unsigned r) {
  return (int)(((unsigned long long)r * s.div_mul) >> s.div_shift);
}

// The places of the tokens t_first, t_first + 1, ..., one per lane, and their exchange.
struct RunPlaces {
  int pos;
  bool ok;
  long long yoff;
  __device__ __forceinline__ void look_up(const TokenMap& tk, const HeadSeg& s, int t_first, int t_last, int lane) {
    pos = 0;
    yoff = 0;
    ok = t_first + lane <= t_last && place_token(tk, s, t_first + lane, pos, yoff);
  }
  __device__ __forceinline__ void take(const RunPlaces& all, int i) {
    pos = __shfl_sync(0xffffffffu, all.pos, i);
    ok = __shfl_sync(0xffffffffu, (int)all.ok, i) != 0;
    yoff = __shfl_sync(0xffffffffu, all.yoff, i);
  }
};

// How a tensor's rows are walked.  ROWS_ANY: a group may straddle tokens.  ROWS_TOKEN: the
// heads fill whole groups, so a group's rows share their token and its turns.  ROWS_FULL: the
// same, with a norm and every dim rotating (no case left to test in the loop).
enum RowsMode { ROWS_ANY, ROWS_TOKEN, ROWS_FULL };
__device__ __forceinline__ int rows_mode(const HeadSeg& s) {
  return s.heads * s.D % 512 != 0 ? ROWS_ANY : s.g && s.inv_freq && s.rotary == s.D ? ROWS_FULL : ROWS_TOKEN;
}

constexpr int NR_STAGES = 4;  // groups in flight per warp
constexpr int NR_GROUP_BYTES = 1024;

// A warp's groups: runs of s.iters consecutive ones, the runs w, w + warps, w + 2 warps, ... of
// the tensor, so that all warps move through memory side by side.
struct WarpRuns {
  int n;          // groups of this warp
  unsigned row0;  // its first row
  __device__ __forceinline__ WarpRuns(const HeadSeg& s, int w, int rpw) {
    const int nruns = (s.groups + s.iters - 1) / s.iters;
    const int mine = w < nruns ? (nruns - 1 - w) / s.warps + 1 : 0;
    n = mine * s.iters;
    if (mine > 0 && w + (mine - 1) * s.warps == nruns - 1) n -= nruns * s.iters - s.groups;
    row0 = (unsigned)w * (unsigned)(s.iters * rpw);
  }
};

// A lane's row as the warp steps through its groups.  SHARED: the heads fill whole groups, so
// all rows of a group belong to one token and, inside a run, the token is found by counting.
// RUNS: the warp goes on to further runs.
template <bool SHARED, bool RUNS, int RPW>
struct RowCursor {
  unsigned r, h;
  int t, left;  // left: groups of the run from this one on
  __device__ __forceinline__ RowCursor(const HeadSeg& s, unsigned row) : r(row), left(s.iters) { find(s); }
  __device__ __forceinline__ void find(const HeadSeg& s) {
    t = row_token(s, r);
    h = r - (unsigned)t * (unsigned)s.heads;
  }
  __device__ __forceinline__ void step(const HeadSeg& s) {
    if (RUNS && --left == 0) {
      left = s.iters;
      r += RPW + (unsigned)(s.warps - 1) * (unsigned)(s.iters * RPW);
      find(s);
      return;
    }
    r += RPW;
    if (SHARED) {
      h += RPW;
      if (h >= (unsigned)s.heads) h -= (unsigned)s.heads, ++t;
    } else {
      find(s);
    }
  }
};

// Looks up the tokens of the run that starts at `row` (`left` groups of the warp from there on);
// returns the first token.
__device__ __forceinline__ int runs_look_up(const TokenMap& tk, const HeadSeg& s, RunPlaces& all, unsigned row, int left,
                                            int rpw, unsigned rows, int lane) {
  const int t_first = row_token(s, row);
  all.look_up(tk, s, t_first, left > 0 ? row_token(s, min(row + (unsigned)(min(s.iters, left) * rpw), rows) - 1) : t_first - 1,
              lane);
  return t_first;
}

// Zeros in the rows of tokens outside the sequences, shared out over `warps` warps.
template <int D>
__device__ __forceinline__ void zero_outside(const TokenMap& tk, const HeadSeg& s, int w, int warps, int lane) {
  const int lo = min(max(tk.cu[0], 0), tk.T), hi = min(max(tk.cu[tk.batch], lo), tk.T);
  const long long n = (long long)(lo + tk.T - hi) * s.heads * (D / 8);
#pragma unroll 1
  for (long long i = w * 32LL + lane; i < n; i += warps * 32LL) {
    const unsigned row = (unsigned)(i / (D / 8));
    const int t = row_token(s, row);
    const int in_token = (int)(row - (unsigned)t * (unsigned)s.heads) * D + (int)(i % (D / 8)) * 8;
    uint16_t* dst = s.y + (long long)(t < lo ? t : t - lo + hi) * s.y_stride + in_token;
    *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D, bool INTER, int MODE>
__device__ __forceinline__ void head_rows_fwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane,
                                              uint8_t* ring, TurnSmem& ts) {
  using L = LaneCols<D, INTER>;
  constexpr bool SHARED = MODE != ROWS_ANY, FULL = MODE == ROWS_FULL;
  constexpr int S = NR_STAGES;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub);
  const bool norm = FULL || s.g != nullptr, turned = FULL || s.inv_freq != nullptr;
  const unsigned rows = (unsigned)p.tk.T * (unsigned)s.heads;
  const int grp0 = warp_in_seg * s.iters, n = min(s.iters, s.groups - grp0);  // one run
  const unsigned row0 = (unsigned)grp0 * L::RPW, row_end = n > 0 ? min(row0 + n * L::RPW, rows) : row0;
  const uint32_t mine = smem_u32(ring) + lane * 16;
  const int de = col.e1 - col.e0;
  RowCursor<SHARED, false, L::RPW> ahead(s, row0 + rg), at = ahead;
  uint32_t fill = 0, use = 0;
  auto issue = [&] {
    if (ahead.r < row_end) {
      const uint16_t* src = s.x + (long long)ahead.t * s.x_stride + (int)(ahead.h * D + col.e0);
      cp_async_16(mine + fill, src, true);
      cp_async_16(mine + fill + 512, src + de, true);
    }
    cp_async_commit();
    ahead.step(s);
    fill = (fill + NR_GROUP_BYTES) & (S * NR_GROUP_BYTES - 1);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  const int t_first = row_token(s, row0), t_last = n > 0 ? row_token(s, row_end - 1) : t_first - 1;
  RunPlaces all, cur;  // looked up while the first rows fly
  all.look_up(p.tk, s, t_first, t_last, lane);
  int cur_t = -1;
  uint4 ga = {}, gb = {};
  if (norm) {
    ga = *reinterpret_cast<const uint4*>(s.g + col.e0);
    gb = *reinterpret_cast<const uint4*>(s.g + col.e1);
  }
  F2 g0[4], g1[4];
  unpack8(ga, g0);
  unpack8(gb, g1);
  load_steps(s, ts);
  LaneTurns turns;
#pragma unroll 2
  for (int it = 0; it < n; ++it) {
    issue();
    const bool in = SHARED || at.r < row_end;
    const int t = in ? at.t : t_last;
    if (SHARED ? t != cur_t : __any_sync(0xffffffffu, t != cur_t)) {
      cur_t = t;
      cur.take(all, t - t_first);
      if (turned) lane_turns<SHARED, FULL>(s, col, ts, cur.pos, turns);
    }
    cp_async_wait<S - 1>();
    const uint8_t* st = ring + lane * 16 + use;
    uint4 xa = *reinterpret_cast<const uint4*>(st), xb = *reinterpret_cast<const uint4*>(st + 512);
    if (norm || turned) {  // else the rows pass as they are
      F2 a[4], b[4];
      unpack8(xa, a);
      unpack8(xb, b);
      if (norm) {
        F2 ss = f2(0.f, 0.f), st2 = ss;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(a[i], a[i], ss), st2 = fma2(b[i], b[i], st2);
        const float2 x = f2_get(ss), y = f2_get(st2);
        const float rstd = rsqrtf(row_sum<L::LPR>((x.x + x.y) + (y.x + y.y)) * (1.f / D) + p.eps);
        const F2 rr = f2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = mul2(mul2(a[i], rr), g0[i]), b[i] = mul2(mul2(b[i], rr), g1[i]);
      }
      rotate16<INTER, false>(a, b, FULL || col.rot0, FULL || col.rot1, turns);
      xa = pack8(a);
      xb = pack8(b);
    }
    if (cur.ok && in) {
      uint16_t* dst = s.y + cur.yoff + (int)(at.h * D + col.e0);
      *reinterpret_cast<uint4*>(dst) = xa;
      *reinterpret_cast<uint4*>(dst + de) = xb;
    }
    at.step(s);
    use = (use + NR_GROUP_BYTES) & (S * NR_GROUP_BYTES - 1);
  }
  cp_async_wait<0>();
}

__device__ __forceinline__ int block_seg(const HeadRowsParams& p) {
  int i = 0;
#pragma unroll
  for (int j = 1; j < NR_MAX_SEGS; ++j)
    if (j < p.nseg && (int)blockIdx.x >= p.seg[j].block0) i = j;
  return i;
}

// D and INTER (0 or 1) of every segment where they agree, else 0 and -1: the call is then
// dispatched per segment, at the registers of the largest form.  ZERO: the blocks from zero_block0
// on write the zeros outside the sequences (a form of its own: in the others the branch alone made
// the append 3 % slower; in the row loops the zeros cost spills).
template <int D, int INTER, bool ZERO>
__global__ void __launch_bounds__(NR_FWD_WARPS * 32, 5) head_rows_fwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) uint8_t rings[NR_FWD_WARPS][NR_STAGES * NR_GROUP_BYTES];
  __shared__ TurnSmem ts;
  const int lane = threadIdx.x % 32;
  if constexpr (ZERO) {
    if ((int)blockIdx.x >= p.zero_block0) {
      const int first = (int)blockIdx.x - p.zero_block0, blocks = (int)gridDim.x - p.zero_block0;
      for (int i = 0; i < p.nseg; ++i)
        zero_outside<D>(p.tk, p.seg[i], first * NR_FWD_WARPS + threadIdx.x / 32, blocks * NR_FWD_WARPS, lane);
      return;
    }
  }
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_FWD_WARPS + threadIdx.x / 32;
  uint8_t* ring = rings[threadIdx.x / 32];
  const int mode = rows_mode(s);
#define DSA_HEAD_ROWS(DD, II)                                                            \
  if ((D == 0 || D == DD) && (INTER < 0 || INTER == II) && s.D == DD && s.interleaved == II) { \
    if (mode == ROWS_FULL) head_rows_fwd<DD, II, ROWS_FULL>(p, s, w, lane, ring, ts);    \
    else if (mode == ROWS_TOKEN) head_rows_fwd<DD, II, ROWS_TOKEN>(p, s, w, lane, ring, ts); \
    else head_rows_fwd<DD, II, ROWS_ANY>(p, s, w, lane, ring, ts);                       \
  }
  DSA_HEAD_ROWS(128, 0) DSA_HEAD_ROWS(128, 1) DSA_HEAD_ROWS(64, 0) DSA_HEAD_ROWS(64, 1) DSA_HEAD_ROWS(32, 0) DSA_HEAD_ROWS(32, 1)
#undef DSA_HEAD_ROWS
}

template <int D, bool INTER, int MODE>
__device__ __forceinline__ void head_rows_bwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane,
                                              uint8_t* ring, TurnSmem& ts, float* acc_smem) {
  using L = LaneCols<D, INTER>;
  constexpr bool SHARED = MODE != ROWS_ANY, FULL = MODE == ROWS_FULL;
  constexpr int S = NR_STAGES;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub);
  const bool norm = FULL || s.g != nullptr, turned = FULL || s.inv_freq != nullptr;
  const unsigned rows = (unsigned)p.tk.T * (unsigned)s.heads;
  const WarpRuns runs(s, warp_in_seg, L::RPW);
  const int n = runs.n;
  const uint32_t mine = smem_u32(ring) + lane * 16;
  const int de = col.e1 - col.e0;
  RowCursor<SHARED, true, L::RPW> ahead(s, runs.row0 + rg), at = ahead;
  int issued = 0;
  uint32_t fill = 0, use = 0;
  auto issue = [&] {
    if (issued < n && (SHARED || ahead.r < rows)) {
      const int in_token = (int)(ahead.h * D + col.e0);
      const uint16_t* src = s.dy + (long long)ahead.t * s.dy_stride + in_token;
      cp_async_16(mine + fill, src, true);
      cp_async_16(mine + fill + 512, src + de, true);
      if (norm) {
        src = s.x + (long long)ahead.t * s.x_stride + in_token;
        cp_async_16(mine + fill + 1024, src, true);
        cp_async_16(mine + fill + 1536, src + de, true);
      }
    }
    cp_async_commit();
    ahead.step(s);
    ++issued;
    fill = (fill + 2 * NR_GROUP_BYTES) & (2 * S * NR_GROUP_BYTES - 1);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  // while the first rows fly (65536 tokens 316 us, as without; before the copies 322, as a call 336)
  if (p.zero_outside) zero_outside<D>(p.tk, s, warp_in_seg, s.warps, lane);
  uint4 ga = {}, gb = {};
  if (norm) {
    ga = *reinterpret_cast<const uint4*>(s.g + col.e0);
    gb = *reinterpret_cast<const uint4*>(s.g + col.e1);
  }
  load_steps(s, ts);
  F2 dg0[4], dg1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dg0[i] = dg1[i] = f2(0.f, 0.f);
  LaneTurns turns;
  RunPlaces all, cur;
  int cur_t = -1, t_first = 0;
#pragma unroll 2
  for (int it = 0; it < n; ++it) {
    if (at.left == s.iters)  // a new run's tokens
      t_first = runs_look_up(p.tk, s, all, at.r - rg, n - it, L::RPW, rows, lane), cur_t = -1;
    issue();
    const bool in = SHARED || at.r < rows;
    const int t = in ? at.t : t_first;
    if (SHARED ? t != cur_t : __any_sync(0xffffffffu, t != cur_t)) {
      cur_t = t;
      cur.take(all, t - t_first);
      if (turned) lane_turns<SHARED, FULL>(s, col, ts, cur.pos, turns);
    }
    const bool ok = cur.ok && in;
    cp_async_wait<S - 1>();
    if (FULL && !ok) {  // the whole group's token
      at.step(s);
      use = (use + 2 * NR_GROUP_BYTES) & (2 * S * NR_GROUP_BYTES - 1);
      continue;
    }
    const uint4* st = reinterpret_cast<const uint4*>(ring + lane * 16 + use);
    F2 a[4], b[4];
    unpack8(st[0], a);
    unpack8(st[32], b);
    rotate16<INTER, true>(a, b, FULL || col.rot0, FULL || col.rot1, turns);  // dn
    if (norm) {
      F2 x0[4], x1[4], g[4], ss = f2(0.f, 0.f), st2 = ss, dot = ss, dot2 = ss, m0[4], m1[4];
      unpack8(st[64], x0);
      unpack8(st[96], x1);
      unpack8(ga, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) m0[i] = mul2(a[i], g[i]), ss = fma2(x0[i], x0[i], ss), dot = fma2(m0[i], x0[i], dot);
      unpack8(gb, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) m1[i] = mul2(b[i], g[i]), st2 = fma2(x1[i], x1[i], st2), dot2 = fma2(m1[i], x1[i], dot2);
      const float2 sa = f2_get(ss), sb = f2_get(st2), da = f2_get(dot), db = f2_get(dot2);
      float sum = (sa.x + sa.y) + (sb.x + sb.y), prod = (da.x + da.y) + (db.x + db.y);
#pragma unroll
      for (int o = 1; o < L::LPR; o <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        prod += __shfl_xor_sync(0xffffffffu, prod, o);
      }
      // dg += dn x rstd;  dx = rstd (dn g - x rstd^2 mean(dn g x))
      const float rstd = rsqrtf(sum * (1.f / D) + p.eps);
      const float back = -(prod * (1.f / D)) * rstd * rstd;
      const F2 rr = f2(rstd, rstd), bb = f2(back, back);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (FULL || ok) {
          dg0[i] = fma2(mul2(a[i], rr), x0[i], dg0[i]);
          dg1[i] = fma2(mul2(b[i], rr), x1[i], dg1[i]);
        }
        a[i] = mul2(rr, fma2(x0[i], bb, m0[i]));
        b[i] = mul2(rr, fma2(x1[i], bb, m1[i]));
      }
    }
    if (ok) {
      uint16_t* dst = s.y + cur.yoff + (int)(at.h * D + col.e0);
      *reinterpret_cast<uint4*>(dst) = pack8(a);
      *reinterpret_cast<uint4*>(dst + de) = pack8(b);
    }
    at.step(s);
    use = (use + 2 * NR_GROUP_BYTES) & (2 * S * NR_GROUP_BYTES - 1);
  }
  cp_async_wait<0>();
  if (!s.g) return;  // block-uniform
  // the block's share of dg: rows of the warp, then the warps in order
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 u = f2_get(dg0[i / 2]), v = f2_get(dg1[i / 2]);
    float x = i & 1 ? u.y : u.x, y = i & 1 ? v.y : v.x;
#pragma unroll
    for (int o = L::LPR; o < 32; o <<= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (rg == 0) {
      acc_smem[warp * D + col.e0 + i] = x;
      acc_smem[warp * D + col.e1 + i] = y;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += NR_BWD_WARPS * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NR_BWD_WARPS; ++w) v += acc_smem[w * D + i];
    s.dg_part[(long long)((int)blockIdx.x - s.block0) * D + i] = v;
  }
}

struct HeadRowsBwdSmem {
  __align__(16) uint8_t rings[NR_BWD_WARPS][NR_STAGES * 2 * NR_GROUP_BYTES];
  TurnSmem ts;
  float acc[NR_BWD_WARPS * 128];
};

template <int D, int INTER>
__global__ void __launch_bounds__(NR_BWD_WARPS * 32, 2) head_rows_bwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  HeadRowsBwdSmem& sm = *reinterpret_cast<HeadRowsBwdSmem*>(smem_raw);
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_BWD_WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* ring = sm.rings[threadIdx.x / 32];
  const int mode = rows_mode(s);
  if (mode == ROWS_FULL) head_rows_bwd<D, INTER, ROWS_FULL>(p, s, w, lane, ring, sm.ts, sm.acc);
  else if (mode == ROWS_TOKEN) head_rows_bwd<D, INTER, ROWS_TOKEN>(p, s, w, lane, ring, sm.ts, sm.acc);
  else head_rows_bwd<D, INTER, ROWS_ANY>(p, s, w, lane, ring, sm.ts, sm.acc);
}

// dg of up to two tensors from their blocks' shares, always in the same order: one block per
// eight dims, 32 strands of shares each.
struct DgParams {
  const float* part[2];
  float* dg[2];
  int blocks[2];
  int D;
};
__global__ void __launch_bounds__(256) head_rows_dg_kernel(const __grid_constant__ DgParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float acc[32][8];
  const int per = p.D / 8, which = blockIdx.x / per, d = (blockIdx.x % per) * 8 + threadIdx.x % 8;
  const int strand = threadIdx.x / 8;
  float v = 0.f;
  for (int i = strand; i < p.blocks[which]; i += 32) v += p.part[which][(long long)i * p.D + d];
  acc[strand][threadIdx.x % 8] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += acc[i][threadIdx.x];
    p.dg[which][d] = sum;
  }
}

}  // namespace dsa

namespace dsa_host {

static long long seg_groups(const dsa::HeadRowsParams& p, const dsa::HeadSeg& s) {
  const long long rpw = 512 / s.D;
  return ((long long)p.tk.T * s.heads + rpw - 1) / rpw;
}
// What a group of a tensor costs, in tenths of one whose turns are at hand: a token's turns
// cost about 4 and are paid once per token and run.
static int group_weight(const dsa::HeadSeg& s) { return 10 + 4 * (512 / s.D) / std::max(s.heads, 512 / s.D); }

// Fills in what the kernels read of each segment: runs of up to `run` groups, of whole tokens
// where `whole` and a token is a few groups, dealt to `total` blocks in all, to the tensors by
// their cost (0: a warp for each run).  Returns the number of blocks.
static int plan_segs(dsa::HeadRowsParams& p, int run, bool whole, long long total, int block_warps) {
  long long cost = 0, block = 0;
  for (int i = 0; i < p.nseg; ++i) cost += seg_groups(p, p.seg[i]) * group_weight(p.seg[i]);
  for (int i = 0; i < p.nseg; ++i) {
    dsa::HeadSeg& s = p.seg[i];
    const int rpw = 512 / s.D;
    s.groups = (int)seg_groups(p, s);
    // consecutive rows touch at most rows / heads + 2 tokens (exactly rows where heads is 1)
    const int token = s.heads % rpw == 0 ? s.heads / rpw : 1;  // groups of a token
    const int mine = whole && token <= 8 ? std::max(run / token, 1) * token : run;
    s.iters = std::min(mine, std::max(1, (s.heads == 1 ? 32 : 30 * s.heads) / rpw));
    int lg = 0;
    while ((1LL << lg) < s.heads) ++lg;
    s.div_shift = 31 + lg;
    s.div_mul = (unsigned)(((1ULL << (31 + lg)) + s.heads - 1) / s.heads);
    s.block0 = (int)block;
    const long long nruns = ((long long)s.groups + s.iters - 1) / s.iters;
    const long long most = (nruns + block_warps - 1) / block_warps, weight = s.groups * (long long)group_weight(s);
    // the nearest share of what is left, which the last tensor takes whole
    const long long share = total ? ((total - block) * weight + cost / 2) / std::max<long long>(cost, 1) : most;
    const long long blocks = std::min(most, std::max<long long>(share, 1));
    cost -= weight;
    s.warps = (int)(blocks * block_warps);
    block += blocks;
  }
  return (int)block;
}

template <bool ZERO>
static int head_rows_fwd_kernel_launch(const dsa::HeadRowsParams& p, int d, int inter, int blocks, cudaStream_t stream) {
  auto kern = d == 128 && inter ? dsa::head_rows_fwd_kernel<128, 1, ZERO>
              : d == 128        ? dsa::head_rows_fwd_kernel<128, 0, ZERO>
              : d == 64 && inter ? dsa::head_rows_fwd_kernel<64, 1, ZERO>
              : d == 64          ? dsa::head_rows_fwd_kernel<64, 0, ZERO>
              : d == 32 && inter ? dsa::head_rows_fwd_kernel<32, 1, ZERO>
              : d == 32          ? dsa::head_rows_fwd_kernel<32, 0, ZERO>
                                 : dsa::head_rows_fwd_kernel<0, -1, false>;
  return launch_pdl(true, kern, dim3((unsigned)blocks), dim3(dsa::NR_FWD_WARPS * 32), 0, stream, p);
}

// Forward: a warp for every run.  Blocks that come and go balance rows of different cost: at
// 32768 tokens of 32 + 4 heads 102 us, against 106 to 142 us in one wave of warps that walk
// many runs, by how the tensors' costs are weighted; an append of as many, 34 against 48 to 58.
// Runs of 8 groups (4: 112 us, 12: 98), fewer where the rows do not fill the SMs otherwise; past
// one and a half waves whole tokens, whose turns are then computed once (1024 tokens: 5.8 us,
// 7.8 without).
int head_rows_fwd_launch(dsa::HeadRowsParams& p, cudaStream_t stream) {
  long long groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += seg_groups(p, p.seg[i]);
  const long long wave = 20LL * sm_count();  // resident warps
  const int run = (int)std::max<long long>(1, std::min<long long>(8, groups / wave));
  int blocks = plan_segs(p, run, 2 * groups > 3 * wave, 0, dsa::NR_FWD_WARPS);
  int d = p.seg[0].D, inter = p.seg[0].interleaved;
  for (int i = 1; i < p.nseg; ++i) {
    if (p.seg[i].D != d || p.seg[i].interleaved != inter) d = 0;
  }
  if (p.zero_outside) {  // (Q and K of one call agree)
    // few of them: at 1024 tokens 148 blocks for the zeros kept the next launch's blocks off the
    // SMs (7.5 us a pass, 5.9 without any or with these)
    p.zero_block0 = blocks;
    blocks += std::min(blocks / 16 + 1, sm_count());
    return head_rows_fwd_kernel_launch<true>(p, d, inter, blocks, stream);
  }
  return head_rows_fwd_kernel_launch<false>(p, d, inter, blocks, stream);
}

// Blocks of the backward: one wave, two blocks on each of a B200's SMs, since each block adds a
// share to the weights' gradients.  They set the order of those sums and the size of the
// workspace, so they follow from the sizes alone and not from the device that is current when
// either is asked for.
static int bwd_plan(dsa::HeadRowsParams& p) {
  const long long blocks = dsa::NR_BWD_BLOCKS;
  long long groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += seg_groups(p, p.seg[i]);
  const long long warps = blocks * dsa::NR_BWD_WARPS;
  const int run = (int)std::max<long long>(1, std::min<long long>(8, (groups + warps - 1) / warps));
  return plan_segs(p, run, false, blocks, dsa::NR_BWD_WARPS);
}
size_t norm_rope_bwd_ws_bytes(long long T, int Hq, int Hk, int d) {
  dsa::HeadRowsParams p{};
  p.tk.T = (int)std::min<long long>(T, INT_MAX);
  for (int H : {Hq, Hk}) {
    if (H == 0) continue;
    p.seg[p.nseg].heads = H;
    p.seg[p.nseg++].D = d;
  }
  return (size_t)bwd_plan(p) * d * sizeof(float);
}
template <int D, int INTER>
static int head_rows_bwd_kernel_launch(const dsa::HeadRowsParams& p, int blocks, cudaStream_t stream) {
  auto kern = dsa::head_rows_bwd_kernel<D, INTER>;
  constexpr int smem = (int)sizeof(dsa::HeadRowsBwdSmem);
  static DeviceFlag attr_done;
  if (!attr_done) {
    if (const cudaError_t e_ = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); e_ != cudaSuccess) return cuda_fail(e_);
    attr_done = true;
  }
  return launch_pdl(true, kern, dim3((unsigned)blocks), dim3(dsa::NR_BWD_WARPS * 32), smem, stream, p);
}

int head_rows_bwd_launch(dsa::HeadRowsParams& p, float* ws, float* const dg[2], cudaStream_t stream) {
  const int blocks = bwd_plan(p);
  dsa::DgParams q{};
  int n = 0;
  for (int i = 0; i < p.nseg; ++i) {
    dsa::HeadSeg& s = p.seg[i];
    s.dg_part = ws + (size_t)s.block0 * s.D;
    if (!s.g) continue;
    q.part[n] = s.dg_part;
    q.dg[n] = dg[i];
    q.blocks[n++] = (i + 1 < p.nseg ? p.seg[i + 1].block0 : blocks) - s.block0;
    q.D = s.D;
  }
  const int d = p.seg[0].D, inter = p.seg[0].interleaved;
  const int st = d == 128 ? (inter ? head_rows_bwd_kernel_launch<128, 1>(p, blocks, stream) : head_rows_bwd_kernel_launch<128, 0>(p, blocks, stream))
                 : d == 64 ? (inter ? head_rows_bwd_kernel_launch<64, 1>(p, blocks, stream) : head_rows_bwd_kernel_launch<64, 0>(p, blocks, stream))
                           : (inter ? head_rows_bwd_kernel_launch<32, 1>(p, blocks, stream) : head_rows_bwd_kernel_launch<32, 0>(p, blocks, stream));
  if (st != DSA_OK || n == 0) return st;
  return launch_pdl(true, dsa::head_rows_dg_kernel, dim3((unsigned)(n * q.D / 8)), dim3(256), 0, stream, q);
}

}  // namespace dsa_host

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
// The angle in turns, position * inv_freq / (2 pi), is formed in fp64 and reduced there to
// [-1/2, 1/2] before it becomes fp32: at position 10^6 an fp32 product would be off by 0.06
// rad, this one by 2e-7 rad.  cos and sin are computed once per token and warp and reused
// over the token's heads.
//
// Layout: D / 16 lanes hold one row, 16 elements each in two 16-byte pieces chosen so that
// both members of a rotation pair sit in the same lane, so the only exchange between lanes
// is the norm's sum (and, backward, its dot product).  A warp takes 512 / D rows at once, a
// group, and runs over consecutive groups: their rows stream through a private ring in shared
// memory by asynchronous copies (no registers held while they fly), and the places of the
// run's tokens (sequence, position, page) are looked up by its lanes side by side, one chain
// of dependent loads per run instead of one per group.
#include <algorithm>

#include "common.cuh"

namespace dsa {

// One tensor of rows: token t's heads are `heads` consecutive rows of D elements.
struct HeadSeg {
  const uint16_t* x;    // [T, heads, D], token stride x_stride (elements)
  const uint16_t* dy;   // backward only: gradient at the output, token stride dy_stride
  uint16_t* y;          // output rows (forward), gradient rows (backward)
  long long x_stride, dy_stride, y_stride;  // y_stride: of a token, or of a page when paged
  const uint16_t* g;    // [D] or null: no norm
  const double* inv_freq;  // [rotary / 2] or null
  int heads, D, rotary;
  int interleaved, paged;
  int block0;           // first block of this tensor's rows
  int groups;           // warp-sized groups of 512 / D rows
  int iters;            // groups of a run (forward: of a warp), at most 32 tokens' worth
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
constexpr int NR_WARPS = 8;

struct HeadRowsParams {
  HeadSeg seg[NR_MAX_SEGS];
  int nseg;
  int warp_iters;  // backward: groups of a warp
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

// cos and sin of pos * inv_freq, the turns reduced in fp64.
__device__ __forceinline__ void turn(double inv_freq, int pos, float& c, float& s) {
  double x = (double)pos * (inv_freq * 0.15915494309189533577);
  x -= rint(x);
  sincospif(2.f * (float)x, &s, &c);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
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

// cos and sin of this lane's eight pairs at its row's position.  Where every row of the warp
// belongs to one token, each of the warp's row groups computes a share and they exchange.
template <int D, bool INTER>
__device__ __forceinline__ void lane_turns(const HeadSeg& s, const LaneCols<D, INTER>& col, bool shared, int rg, int pos,
                                           float* c, float* sn) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  constexpr int PER = RPW >= 8 ? 1 : 8 / RPW;  // pairs per row group when shared
  if (shared) {
    float mc[PER], ms[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int p = (rg * PER + j) & 7;
      mc[j] = 1.f, ms[j] = 0.f;
      if (col.rotates(p)) turn(s.inv_freq[col.freq(p)], pos, mc[j], ms[j]);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int src = (p / PER) * LPR + col.sub;
      c[p] = __shfl_sync(0xffffffffu, mc[p % PER], src);
      sn[p] = __shfl_sync(0xffffffffu, ms[p % PER], src);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      c[p] = 1.f, sn[p] = 0.f;
      if (col.rotates(p)) turn(s.inv_freq[col.freq(p)], pos, c[p], sn[p]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Pair rotation of the lane's 16 values (two pieces) by the angles (c, sgn * sn).
template <bool INTER>
__device__ __forceinline__ void rotate16(float* a, float* b, bool rot0, bool rot1, const float* c, const float* sn, float sgn) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (!(half ? rot1 : rot0)) continue;  // dims that pass stay out of every product
#pragma unroll
    for (int p = 4 * half; p < 4 * half + 4; ++p) {
      float& u = INTER ? (p < 4 ? a[2 * (p & 3)] : b[2 * (p & 3)]) : a[p];
      float& v = INTER ? (p < 4 ? a[2 * (p & 3) + 1] : b[2 * (p & 3) + 1]) : b[p];
      const float s = sgn * sn[p], u0 = u, v0 = v;
      u = fmaf(u0, c[p], -(v0 * s));
      v = fmaf(v0, c[p], u0 * s);
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

constexpr int NR_FWD_STAGES = 4;  // groups in flight per warp
constexpr int NR_GROUP_BYTES = 1024;

template <int D, bool INTER>
__device__ __forceinline__ void head_rows_fwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane,
                                              uint8_t* ring) {
  using L = LaneCols<D, INTER>;
  constexpr int S = NR_FWD_STAGES;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub);
  const unsigned H = s.heads;
  const bool shared = H % L::RPW == 0;
  const unsigned rows = (unsigned)p.tk.T * H;
  const int grp0 = warp_in_seg * s.iters, n = min(s.iters, s.groups - grp0);
  if (n <= 0) return;
  const unsigned row0 = (unsigned)grp0 * L::RPW;
  uint8_t* mine = ring + lane * 16;
  auto issue = [&](int it) {
    const unsigned r = row0 + it * L::RPW + rg;
    if (it < n && r < rows) {
      const int t = row_token(s, r);
      const uint16_t* src = s.x + (long long)t * s.x_stride + (r - (unsigned)t * H) * D;
      const uint32_t dst = smem_u32(mine + (it % S) * NR_GROUP_BYTES);
      cp_async_16(dst, src + col.e0, true);
      cp_async_16(dst + 512, src + col.e1, true);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  const int t_first = row_token(s, row0), t_last = row_token(s, min(row0 + n * L::RPW, rows) - 1);
  RunPlaces all, cur;
  all.look_up(p.tk, s, t_first, t_last, lane);
  uint4 ga = {}, gb = {};
  if (s.g) {
    ga = *reinterpret_cast<const uint4*>(s.g + col.e0);
    gb = *reinterpret_cast<const uint4*>(s.g + col.e1);
  }
  float g0[8], g1[8];
  unpack8(ga, g0);
  unpack8(gb, g1);
  float c[8], sn[8];
  int cur_t = -1;
#pragma unroll 1
  for (int it = 0; it < n; ++it) {
    issue(it + S - 1);
    const unsigned r = row0 + it * L::RPW + rg;
    const int t = r < rows ? row_token(s, r) : t_last;
    const unsigned h = r - (unsigned)t * H;
    if (__any_sync(0xffffffffu, t != cur_t)) {
      cur_t = t;
      cur.take(all, t - t_first);
      if (s.inv_freq) lane_turns(s, col, shared, rg, cur.pos, c, sn);
    }
    cp_async_wait<S - 1>();
    uint4 xa = *reinterpret_cast<const uint4*>(mine + (it % S) * NR_GROUP_BYTES);
    uint4 xb = *reinterpret_cast<const uint4*>(mine + (it % S) * NR_GROUP_BYTES + 512);
    if (s.g || s.inv_freq) {  // else the rows pass as they are
      float a[8], b[8];
      unpack8(xa, a);
      unpack8(xb, b);
      if (s.g) {
        float ss = 0.f, st = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss), st = fmaf(b[i], b[i], st);
        const float rstd = rsqrtf(row_sum<L::LPR>(ss + st) * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] *= rstd * g0[i];
          b[i] *= rstd * g1[i];
        }
      }
      rotate16<INTER>(a, b, col.rot0, col.rot1, c, sn, 1.f);
      xa = pack8(a);
      xb = pack8(b);
    }
    if (cur.ok && r < rows) {
      uint16_t* dst = s.y + cur.yoff + h * D;
      *reinterpret_cast<uint4*>(dst + col.e0) = xa;
      *reinterpret_cast<uint4*>(dst + col.e1) = xb;
    }
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

__global__ void __launch_bounds__(NR_WARPS * 32, 3) head_rows_fwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) uint8_t rings[NR_WARPS][NR_FWD_STAGES * NR_GROUP_BYTES];
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* ring = rings[threadIdx.x / 32];
  if (s.interleaved) {
    if (s.D == 128) head_rows_fwd<128, true>(p, s, w, lane, ring);
    else if (s.D == 64) head_rows_fwd<64, true>(p, s, w, lane, ring);
    else head_rows_fwd<32, true>(p, s, w, lane, ring);
  } else {
    if (s.D == 128) head_rows_fwd<128, false>(p, s, w, lane, ring);
    else if (s.D == 64) head_rows_fwd<64, false>(p, s, w, lane, ring);
    else head_rows_fwd<32, false>(p, s, w, lane, ring);
  }
}

constexpr int NR_BWD_STAGES = 3;  // groups in flight per warp, of x and of dy

template <int D, bool INTER>
__device__ __forceinline__ void head_rows_bwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane,
                                              uint8_t* ring, float* acc_smem) {
  using L = LaneCols<D, INTER>;
  constexpr int S = NR_BWD_STAGES;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub);
  const unsigned H = s.heads;
  const bool shared = H % L::RPW == 0;
  const unsigned rows = (unsigned)p.tk.T * H;
  const int grp0 = (int)min((long long)warp_in_seg * p.warp_iters, (long long)s.groups);
  const int n = min(p.warp_iters, s.groups - grp0);
  const unsigned row0 = (unsigned)grp0 * L::RPW;
  uint8_t* mine = ring + lane * 16;
  auto issue = [&](int it) {
    const unsigned r = row0 + it * L::RPW + rg;
    if (it < n && r < rows) {
      const int t = row_token(s, r);
      const unsigned h = r - (unsigned)t * H;
      const uint32_t dst = smem_u32(mine + (it % S) * 2 * NR_GROUP_BYTES);
      const uint16_t* src = s.dy + (long long)t * s.dy_stride + h * D;
      cp_async_16(dst, src + col.e0, true);
      cp_async_16(dst + 512, src + col.e1, true);
      if (s.g) {
        src = s.x + (long long)t * s.x_stride + h * D;
        cp_async_16(dst + 1024, src + col.e0, true);
        cp_async_16(dst + 1536, src + col.e1, true);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  uint4 ga = {}, gb = {};
  if (s.g) {
    ga = *reinterpret_cast<const uint4*>(s.g + col.e0);
    gb = *reinterpret_cast<const uint4*>(s.g + col.e1);
  }
  float dg0[8] = {}, dg1[8] = {}, c[8], sn[8];
  RunPlaces all, cur;
  int cur_t = -1, t_first = 0, run_end = 0;
#pragma unroll 1
  for (int it = 0; it < n; ++it) {
    if (it == run_end) {  // the next run's tokens
      run_end = min(it + s.iters, n);
      t_first = row_token(s, row0 + it * L::RPW);
      all.look_up(p.tk, s, t_first, row_token(s, min(row0 + run_end * L::RPW, rows) - 1), lane);
    }
    issue(it + S - 1);
    const unsigned r = row0 + it * L::RPW + rg;
    const bool in = r < rows;
    const int t = in ? row_token(s, r) : t_first;
    const unsigned h = r - (unsigned)t * H;
    if (__any_sync(0xffffffffu, t != cur_t)) {
      cur_t = t;
      cur.take(all, t - t_first);
      if (s.inv_freq) lane_turns(s, col, shared, rg, cur.pos, c, sn);
    }
    const bool ok = cur.ok && in;
    cp_async_wait<S - 1>();
    const uint4* st = reinterpret_cast<const uint4*>(mine + (it % S) * 2 * NR_GROUP_BYTES);
    float a[8], b[8];
    unpack8(st[0], a);
    unpack8(st[32], b);
    rotate16<INTER>(a, b, col.rot0, col.rot1, c, sn, -1.f);
    if (s.g) {
      float xf[8], xg[8], g[8];
      unpack8(st[64], xf);
      unpack8(st[96], xg);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(xf[i], xf[i], fmaf(xg[i], xg[i], ss));
      const float rstd = rsqrtf(row_sum<L::LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) xf[i] *= rstd, xg[i] *= rstd;  // xh
      if (ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dg0[i] = fmaf(a[i], xf[i], dg0[i]), dg1[i] = fmaf(b[i], xg[i], dg1[i]);
      }
      unpack8(ga, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] *= g[i], dot = fmaf(a[i], xf[i], dot);
      unpack8(gb, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] *= g[i], dot = fmaf(b[i], xg[i], dot);
      const float mean = row_sum<L::LPR>(dot) * (1.f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = rstd * fmaf(-xf[i], mean, a[i]);
        b[i] = rstd * fmaf(-xg[i], mean, b[i]);
      }
    }
    if (ok) {
      uint16_t* dst = s.y + cur.yoff + h * D;
      *reinterpret_cast<uint4*>(dst + col.e0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + col.e1) = pack8(b);
    }
  }
  cp_async_wait<0>();
  if (!s.g) return;  // block-uniform
  // the block's share of dg: rows of the warp, then the warps in order
#pragma unroll
  for (int o = L::LPR; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dg0[i] += __shfl_xor_sync(0xffffffffu, dg0[i], o);
      dg1[i] += __shfl_xor_sync(0xffffffffu, dg1[i], o);
    }
  const int warp = threadIdx.x / 32;
  if (rg == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc_smem[warp * D + col.e0 + i] = dg0[i];
      acc_smem[warp * D + col.e1 + i] = dg1[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += NR_WARPS * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NR_WARPS; ++w) v += acc_smem[w * D + i];
    s.dg_part[(long long)((int)blockIdx.x - s.block0) * D + i] = v;
  }
}

struct HeadRowsBwdSmem {
  __align__(16) uint8_t rings[NR_WARPS][NR_BWD_STAGES * 2 * NR_GROUP_BYTES];
  float acc[NR_WARPS * 128];
};

__global__ void __launch_bounds__(NR_WARPS * 32, 2) head_rows_bwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  HeadRowsBwdSmem& sm = *reinterpret_cast<HeadRowsBwdSmem*>(smem_raw);
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* ring = sm.rings[threadIdx.x / 32];
  if (s.interleaved) {
    if (s.D == 128) head_rows_bwd<128, true>(p, s, w, lane, ring, sm.acc);
    else if (s.D == 64) head_rows_bwd<64, true>(p, s, w, lane, ring, sm.acc);
    else head_rows_bwd<32, true>(p, s, w, lane, ring, sm.acc);
  } else {
    if (s.D == 128) head_rows_bwd<128, false>(p, s, w, lane, ring, sm.acc);
    else if (s.D == 64) head_rows_bwd<64, false>(p, s, w, lane, ring, sm.acc);
    else head_rows_bwd<32, false>(p, s, w, lane, ring, sm.acc);
  }
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
// Fills in what the kernels read of each segment; a warp takes warp_iters groups, or where
// that is 0 as many as make a run.  Returns the number of blocks.
static int plan_segs(dsa::HeadRowsParams& p, int run, int warp_iters) {
  long long block = 0;
  for (int i = 0; i < p.nseg; ++i) {
    dsa::HeadSeg& s = p.seg[i];
    const int rpw = 512 / s.D;
    s.groups = (int)seg_groups(p, s);
    // consecutive rows touch at most rows / heads + 2 tokens (exactly rows where heads is 1)
    s.iters = std::min(run, std::max(1, (s.heads == 1 ? 32 : 30 * s.heads) / rpw));
    int lg = 0;
    while ((1LL << lg) < s.heads) ++lg;
    s.div_shift = 31 + lg;
    s.div_mul = (unsigned)(((1ULL << (31 + lg)) + s.heads - 1) / s.heads);
    s.block0 = (int)block;
    const long long per_block = (long long)(warp_iters ? warp_iters : s.iters) * dsa::NR_WARPS;
    block += (s.groups + per_block - 1) / per_block;
  }
  return (int)block;
}

int head_rows_fwd_launch(dsa::HeadRowsParams& p, bool pdl, cudaStream_t stream) {
  long long groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += seg_groups(p, p.seg[i]);
  const int blocks = plan_segs(p, groups > 32LL * sm_count() ? 8 : 1, 0);
  return launch_pdl(pdl, dsa::head_rows_fwd_kernel, dim3((unsigned)blocks), dim3(dsa::NR_WARPS * 32), 0, stream, p);
}

// Groups per warp of the backward: the whole call in at most 16 warps' worth per SM.
static int bwd_iters(long long groups) {
  const long long warps = 16LL * sm_count();
  return (int)std::max<long long>(1, (groups + warps - 1) / warps);
}
size_t norm_rope_bwd_ws_bytes(long long T, int Hq, int Hk, int d) {
  const long long rpw = 512 / d, nq = (T * Hq + rpw - 1) / rpw, nk = (T * Hk + rpw - 1) / rpw;
  const long long per_block = (long long)bwd_iters(nq + nk) * dsa::NR_WARPS;
  return (size_t)((nq + per_block - 1) / per_block + (nk + per_block - 1) / per_block) * d * sizeof(float);
}
int head_rows_bwd_launch(dsa::HeadRowsParams& p, float* ws, float* const dg[2], cudaStream_t stream) {
  long long groups = 0;
  for (int i = 0; i < p.nseg; ++i) groups += seg_groups(p, p.seg[i]);
  p.warp_iters = bwd_iters(groups);
  const int blocks = plan_segs(p, 8, p.warp_iters);
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
  static DeviceFlag attr_done;
  if (!attr_done) {
    if (const cudaError_t e_ = cudaFuncSetAttribute(dsa::head_rows_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    (int)sizeof(dsa::HeadRowsBwdSmem));
        e_ != cudaSuccess)
      return cuda_fail(e_);
    attr_done = true;
  }
  if (const int st = launch_pdl(false, dsa::head_rows_bwd_kernel, dim3((unsigned)blocks), dim3(dsa::NR_WARPS * 32),
                                sizeof(dsa::HeadRowsBwdSmem), stream, p);
      st != DSA_OK || n == 0)
    return st;
  return launch_pdl(true, dsa::head_rows_dg_kernel, dim3((unsigned)(n * q.D / 8)), dim3(256), 0, stream, q);
}

}  // namespace dsa_host

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
// is the norm's sum (and, backward, its dot product).  A warp takes 512 / D rows at once.
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
  int iters;  // groups per warp
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

// What a lane holds of every row of its segment: two 8-element pieces at e0 and e1.
template <int D>
struct LaneCols {
  static constexpr int LPR = D / 16;       // lanes per row
  static constexpr int RPW = 32 / LPR;     // rows per warp
  int e0, e1;
  bool rot;  // this lane's pairs rotate (frequencies 8 sub .. 8 sub + 7)

  __device__ __forceinline__ LaneCols(const HeadSeg& s, int sub, bool inter) {
    const int nrot = s.inv_freq ? s.rotary / 16 : 0;  // rotating lanes
    rot = sub < nrot;
    if (inter) {
      e0 = 16 * sub;
      e1 = e0 + 8;
    } else if (rot) {
      e0 = 8 * sub;
      e1 = 8 * (sub + nrot);
    } else {
      e0 = 16 * sub;  // pieces 2 nrot + 2 (sub - nrot) and the next
      e1 = e0 + 8;
    }
  }
};

// cos and sin of this lane's eight pairs at its row's position.  Where every row of the warp
// belongs to one token, each of the warp's row groups computes a share and they exchange.
template <int D>
__device__ __forceinline__ void lane_turns(const HeadSeg& s, bool shared, bool rot, int sub, int rg, int pos, float* c,
                                           float* sn) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  constexpr int PER = RPW >= 8 ? 1 : 8 / RPW;  // pairs per row group when shared
  if (shared) {
    float mc[PER], ms[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int p = (rg * PER + j) & 7;
      if (rot) turn(s.inv_freq[8 * sub + p], pos, mc[j], ms[j]);
      else mc[j] = 1.f, ms[j] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int src = (p / PER) * LPR + sub;
      c[p] = __shfl_sync(0xffffffffu, mc[p % PER], src);
      sn[p] = __shfl_sync(0xffffffffu, ms[p % PER], src);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (rot) turn(s.inv_freq[8 * sub + p], pos, c[p], sn[p]);
      else c[p] = 1.f, sn[p] = 0.f;
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
__device__ __forceinline__ void rotate16(float* a, float* b, const float* c, const float* sn, float sgn) {
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float& u = INTER ? (p < 4 ? a[2 * (p & 3)] : b[2 * (p & 3)]) : a[p];
    float& v = INTER ? (p < 4 ? a[2 * (p & 3) + 1] : b[2 * (p & 3) + 1]) : b[p];
    const float s = sgn * sn[p], u0 = u, v0 = v;
    u = fmaf(u0, c[p], -(v0 * s));
    v = fmaf(v0, c[p], u0 * s);
  }
}

template <int D, bool INTER>
__device__ __forceinline__ void head_rows_fwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane) {
  using L = LaneCols<D>;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub, INTER);
  const unsigned H = s.heads;
  const bool shared = H % L::RPW == 0;
  const unsigned rows = (unsigned)p.tk.T * H;
  float g0[8], g1[8];
  if (s.g) {
    unpack8(*reinterpret_cast<const uint4*>(s.g + col.e0), g0);
    unpack8(*reinterpret_cast<const uint4*>(s.g + col.e1), g1);
  }
  float c[8], sn[8];
  int cur = -1;
  bool ok = false;
  long long yoff = 0;
  for (int it = 0; it < p.iters; ++it) {
    const int grp = warp_in_seg * p.iters + it;
    if (grp >= s.groups) break;  // warp-uniform
    const unsigned r = (unsigned)grp * L::RPW + rg;
    const int t = r < rows ? (int)(r / H) : p.tk.T;
    const unsigned h = r - (unsigned)t * H;
    uint4 xa = {}, xb = {};
    if (r < rows) {
      const uint16_t* src = s.x + (long long)t * s.x_stride + h * D;
      xa = *reinterpret_cast<const uint4*>(src + col.e0);
      xb = *reinterpret_cast<const uint4*>(src + col.e1);
    }
    if (__any_sync(0xffffffffu, t != cur)) {
      cur = t;
      int pos = 0;
      ok = place_token(p.tk, s, t, pos, yoff);
      if (s.inv_freq) lane_turns<D>(s, shared, col.rot, sub, rg, pos, c, sn);
    }
    float a[8], b[8];
    unpack8(xa, a);
    unpack8(xb, b);
    if (s.g) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
      const float rstd = rsqrtf(row_sum<L::LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= rstd * g0[i];
        b[i] *= rstd * g1[i];
      }
    }
    if (s.inv_freq && col.rot) rotate16<INTER>(a, b, c, sn, 1.f);
    if (ok) {
      uint16_t* dst = s.y + yoff + h * D;
      *reinterpret_cast<uint4*>(dst + col.e0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + col.e1) = pack8(b);
    }
  }
}

__device__ __forceinline__ int block_seg(const HeadRowsParams& p) {
  int i = 0;
#pragma unroll
  for (int j = 1; j < NR_MAX_SEGS; ++j)
    if (j < p.nseg && (int)blockIdx.x >= p.seg[j].block0) i = j;
  return i;
}

__global__ void __launch_bounds__(NR_WARPS * 32) head_rows_fwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (s.interleaved) {
    if (s.D == 128) head_rows_fwd<128, true>(p, s, w, lane);
    else if (s.D == 64) head_rows_fwd<64, true>(p, s, w, lane);
    else head_rows_fwd<32, true>(p, s, w, lane);
  } else {
    if (s.D == 128) head_rows_fwd<128, false>(p, s, w, lane);
    else if (s.D == 64) head_rows_fwd<64, false>(p, s, w, lane);
    else head_rows_fwd<32, false>(p, s, w, lane);
  }
}

template <int D, bool INTER>
__device__ __forceinline__ void head_rows_bwd(const HeadRowsParams& p, const HeadSeg& s, int warp_in_seg, int lane,
                                              float* acc_smem) {
  using L = LaneCols<D>;
  const int sub = lane % L::LPR, rg = lane / L::LPR;
  const L col(s, sub, INTER);
  const unsigned H = s.heads;
  const bool shared = H % L::RPW == 0;
  const unsigned rows = (unsigned)p.tk.T * H;
  float g0[8], g1[8], dg0[8] = {}, dg1[8] = {};
  if (s.g) {
    unpack8(*reinterpret_cast<const uint4*>(s.g + col.e0), g0);
    unpack8(*reinterpret_cast<const uint4*>(s.g + col.e1), g1);
  }
  float c[8], sn[8];
  int cur = -1;
  bool ok = false;
  long long yoff = 0;
  for (int it = 0; it < p.iters; ++it) {
    const int grp = warp_in_seg * p.iters + it;
    if (grp >= s.groups) break;  // warp-uniform
    const unsigned r = (unsigned)grp * L::RPW + rg;
    const int t = r < rows ? (int)(r / H) : p.tk.T;
    const unsigned h = r - (unsigned)t * H;
    uint4 xa = {}, xb = {}, ya = {}, yb = {};
    if (r < rows) {
      const uint16_t* src = s.dy + (long long)t * s.dy_stride + h * D;
      ya = *reinterpret_cast<const uint4*>(src + col.e0);
      yb = *reinterpret_cast<const uint4*>(src + col.e1);
      if (s.g) {
        src = s.x + (long long)t * s.x_stride + h * D;
        xa = *reinterpret_cast<const uint4*>(src + col.e0);
        xb = *reinterpret_cast<const uint4*>(src + col.e1);
      }
    }
    if (__any_sync(0xffffffffu, t != cur)) {
      cur = t;
      int pos = 0;
      ok = place_token(p.tk, s, t, pos, yoff);
      if (s.inv_freq) lane_turns<D>(s, shared, col.rot, sub, rg, pos, c, sn);
    }
    float a[8], b[8];
    unpack8(ya, a);
    unpack8(yb, b);
    if (s.inv_freq && col.rot) rotate16<INTER>(a, b, c, sn, -1.f);
    if (s.g) {
      float xf[8], xg[8];
      unpack8(xa, xf);
      unpack8(xb, xg);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(xf[i], xf[i], fmaf(xg[i], xg[i], ss));
        dot = fmaf(a[i] * g0[i], xf[i], fmaf(b[i] * g1[i], xg[i], dot));
      }
      const float rstd = rsqrtf(row_sum<L::LPR>(ss) * (1.f / D) + p.eps);
      const float mean = row_sum<L::LPR>(dot) * rstd * (1.f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h0 = xf[i] * rstd, h1 = xg[i] * rstd;
        if (ok) {
          dg0[i] = fmaf(a[i], h0, dg0[i]);
          dg1[i] = fmaf(b[i], h1, dg1[i]);
        }
        a[i] = rstd * (a[i] * g0[i] - h0 * mean);
        b[i] = rstd * (b[i] * g1[i] - h1 * mean);
      }
    }
    if (ok) {
      uint16_t* dst = s.y + yoff + h * D;
      *reinterpret_cast<uint4*>(dst + col.e0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + col.e1) = pack8(b);
    }
  }
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

__global__ void __launch_bounds__(NR_WARPS * 32) head_rows_bwd_kernel(const __grid_constant__ HeadRowsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float acc[NR_WARPS * 128];
  const HeadSeg& s = p.seg[block_seg(p)];
  const int w = ((int)blockIdx.x - s.block0) * NR_WARPS + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (s.interleaved) {
    if (s.D == 128) head_rows_bwd<128, true>(p, s, w, lane, acc);
    else if (s.D == 64) head_rows_bwd<64, true>(p, s, w, lane, acc);
    else head_rows_bwd<32, true>(p, s, w, lane, acc);
  } else {
    if (s.D == 128) head_rows_bwd<128, false>(p, s, w, lane, acc);
    else if (s.D == 64) head_rows_bwd<64, false>(p, s, w, lane, acc);
    else head_rows_bwd<32, false>(p, s, w, lane, acc);
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
__global__ void __launch_bounds__(256) head_rows_dg_kernel(const DgParams p) {
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

static void head_seg_blocks(dsa::HeadRowsParams& p) {
  int block = 0;
  for (int i = 0; i < p.nseg; ++i) {
    dsa::HeadSeg& s = p.seg[i];
    const long long rows = (long long)p.tk.T * s.heads, rpw = 512 / s.D;
    s.groups = (int)((rows + rpw - 1) / rpw);
    s.block0 = block;
    const long long per_block = (long long)p.iters * dsa::NR_WARPS;
    block += (int)((s.groups + per_block - 1) / per_block);
  }
}
static int head_rows_blocks(const dsa::HeadRowsParams& p) {
  const dsa::HeadSeg& s = p.seg[p.nseg - 1];
  const long long per_block = (long long)p.iters * dsa::NR_WARPS;
  return s.block0 + (int)((s.groups + per_block - 1) / per_block);
}
static long long head_rows_groups(const dsa::HeadRowsParams& p) {
  long long n = 0;
  for (int i = 0; i < p.nseg; ++i) n += ((long long)p.tk.T * p.seg[i].heads + 512 / p.seg[i].D - 1) / (512 / p.seg[i].D);
  return n;
}

int head_rows_fwd_launch(dsa::HeadRowsParams& p, bool pdl, cudaStream_t stream) {
  p.iters = head_rows_groups(p) > 32LL * sm_count() ? 8 : 1;
  head_seg_blocks(p);
  return launch_pdl(pdl, dsa::head_rows_fwd_kernel, dim3((unsigned)head_rows_blocks(p)), dim3(dsa::NR_WARPS * 32), 0,
                    stream, p);
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
  p.iters = bwd_iters(head_rows_groups(p));
  head_seg_blocks(p);
  const int blocks = head_rows_blocks(p);
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
  if (const int st = launch_pdl(false, dsa::head_rows_bwd_kernel, dim3((unsigned)blocks), dim3(dsa::NR_WARPS * 32), 0,
                                stream, p);
      st != DSA_OK || n == 0)
    return st;
  return launch_pdl(true, dsa::head_rows_dg_kernel, dim3((unsigned)(n * q.D / 8)), dim3(256), 0, stream, q);
}

}  // namespace dsa_host

// Attention of one query row per sequence over its selected positions in a paged key and
// value cache (sm_100a).
//
//   O[b, h, :] = sum_{s in S_b} softmax_s(scale * Q[b, h, :] . K[s, g, :]) V[s, g, :],  g = h / (Hq / Hkv)
//
// S_b: the entries of indices[b, :] inside [0, len_b) whose page lies in the pool; position s
// is row s mod P of page table[b, s / P].  An empty set gives O = 0 and lse = -inf.
//
// The work is a gather of 2 Hkv d bf16 per selected position; the products are 16 operations
// per byte, so warp-level MMA carries them (16 keys x 8 heads, no padding) as in the gather
// kernel of the contiguous cache.  One launch and no scratch memory: the selected slots of a
// (row, KV head) are dealt 32 at a time to the warps of a thread-block cluster, each warp runs
// one online softmax over its slots, 16 at a time, and the partial (max, sum, O) of the warps
// are joined in shared memory, then over the cluster: each block sends its share of every
// output to the block that finishes it (remote stores, one barrier, local sums), always summed
// in the same order.
#include <algorithm>
#include <cooperative_groups.h>

#include "common.cuh"
#include "warp_mma.cuh"

namespace dsa {

struct SAPagedParams {
  const uint16_t* Q;  // [rows, Hq, D]
  const uint16_t* K;  // [pages, P, Hkv, D], page strides below (elements)
  const uint16_t* V;
  long long k_page_stride, v_page_stride;
  const int* indices;  // [rows, k]
  const int* table;    // [rows, table_width]
  const int* lens;     // [rows]
  int table_width, page_shift, num_pages;
  int Hq, Hkv, G, k;
  float scale_log2;
  uint16_t* O;  // [rows, Hq, D]
  float* lse;   // [rows, Hq] or null
};

constexpr int SAP_MAX_SPLITS = 8;  // blocks of a cluster (the portable limit)

template <int D, int WARPS, int STAGES>
struct SAPagedSmem {
  static constexpr int STAGE_BYTES = 2 * 16 * D * 2;  // K and V rows of a chunk
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int OFF_ML = RING;                    // [WARPS][8] float4: max, sum, rounded sum
  // what the cluster's blocks send to this one: the states of all of them, and their O of the
  // outputs that this block finishes (outputs rank, rank + splits, ... of the 8 D)
  static constexpr int OFF_CML = OFF_ML + WARPS * 8 * 16;             // [splits][8] float4
  static constexpr int OFF_CO = OFF_CML + SAP_MAX_SPLITS * 8 * 16;    // [splits][ceil(8 D / splits)]
  static constexpr int BYTES = OFF_CO + (8 * D + SAP_MAX_SPLITS) * 4;
  static_assert(STAGES * STAGE_BYTES >= 8 * D * 4, "a warp's O replaces its ring");
};

template <int D, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32) sparse_attn_paged_kernel(const SAPagedParams p, int splits) {
  namespace cg = cooperative_groups;
  using C = SAPagedSmem<D, WARPS, STAGES>;
  constexpr int SEGS = D / 8, MT = D / 16;
  constexpr int TILE_BYTES = C::STAGE_BYTES / 2;
  pdl_wait();
  pdl_trigger();
  if (splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* my = smem + warp * STAGES * C::STAGE_BYTES;
  const uint32_t my_s = smem_u32(my);
  const int rank = blockIdx.x % splits, cid = blockIdx.x / splits;
  const int g = cid % p.Hkv;
  const long long row = cid / p.Hkv;

  const int* idx = p.indices + row * p.k;
  const int* trow = p.table + row * p.table_width;
  const int nunits = (p.k + 31) / 32, step = splits * WARPS, u0 = rank * WARPS + warp;
  const int nchunks = u0 < nunits ? 2 * ((nunits - 1 - u0) / step + 1) : 0;  // of this warp
  const int kv_row = p.Hkv * D;
  const uint16_t* Kg = p.K + g * D;
  const uint16_t* Vg = p.V + g * D;

  const int len = __ldg(p.lens + row);
  uint32_t qb[MT][2];
  {
    const int head = lane / 4;
    const bool hv = head < p.G;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.Q + ((size_t)row * p.Hq + g * p.G + (hv ? head : 0)) * D);
#pragma unroll
    for (int kk = 0; kk < MT; ++kk) {
      qb[kk][0] = hv ? __ldg(qrow + kk * 8 + (lane % 4)) : 0u;
      qb[kk][1] = hv ? __ldg(qrow + kk * 8 + 4 + (lane % 4)) : 0u;
    }
  }

  // Slots are handled 32 at a time, a unit, one per lane: two chunks.  The chain position ->
  // page -> row is three dependent loads, so a unit's pages are looked up one unit ahead of its
  // copies and its positions two ahead.
  auto position = [&](int u) { return u < nunits && u * 32 + lane < p.k ? __ldg(idx + u * 32 + lane) : -1; };
  // cache slot (page * P + row in page) of a position, or -1
  auto cache_slot = [&](int s) {
    if ((unsigned)s >= (unsigned)max(len, 0)) return -1;
    const int pg = s >> p.page_shift;
    if (pg >= p.table_width) return -1;
    const int page = __ldg(trow + pg);
    if ((unsigned)page >= (unsigned)p.num_pages) return -1;
    return (page << p.page_shift) | (s & ((1 << p.page_shift) - 1));
  };
  // starts the copies of a chunk, the lanes' slots from `first` on; returns its mask of valid slots
  auto issue = [&](int st, int mine, int first) -> uint32_t {
    const uint32_t kdst = my_s + st * C::STAGE_BYTES, vdst = kdst + TILE_BYTES;
    const int sub = lane >> 3, c = lane & 7;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + sub;
      const int cs = __shfl_sync(0xffffffffu, mine, first + r);
      const bool valid = cs >= 0;
      const int page = cs >> p.page_shift;
      const int in = (cs & ((1 << p.page_shift) - 1)) * kv_row + c * 8;
      const uint16_t* ksrc = valid ? Kg + page * p.k_page_stride + in : Kg;
      const uint16_t* vsrc = valid ? Vg + page * p.v_page_stride + in : Vg;
      const uint32_t o = tile_off<D>(r, c);
#pragma unroll
      for (int h = 0; h < SEGS / 8; ++h) {
        cp_async_16(kdst + o + h * 128, ksrc + h * 64, valid);
        cp_async_16(vdst + o + h * 128, vsrc + h * 64, valid);
      }
    }
    cp_async_commit();
    return (__ballot_sync(0xffffffffu, mine >= 0) >> first) & 0xFFFFu;
  };

  float acc[MT][4] = {};
  float m0 = -INFINITY, m1 = -INFINITY;  // running max (log2 domain) of heads h0, h1
  float l0 = 0.f, l1 = 0.f;              // this lane's share of the sums (for the lse)
  float r0 = 0.f, r1 = 0.f;              // the same of the bf16-rounded weights that multiply V

  uint32_t vmr[STAGES];  // valid masks of the chunks in flight, the next one to use first
  int cs_cur = -1, cs_next, s_next, u_next = u0 + step;
  {
    const int s0 = position(u0), s1 = position(u_next);
    cs_cur = cache_slot(s0);
    cs_next = cache_slot(s1);
    s_next = position(u_next += step);
  }
  auto issue_chunk = [&](int n) -> uint32_t {
    if (n >= nchunks) {
      cp_async_commit();
      return 0u;
    }
    if (n > 0 && n % 2 == 0) {  // the next unit
      cs_cur = cs_next;
      cs_next = cache_slot(s_next);
      s_next = position(u_next += step);
    }
    return issue(n % STAGES, cs_cur, n % 2 * 16);
  };
#pragma unroll
  for (int j = 0; j < STAGES - 1; ++j) vmr[j] = issue_chunk(j);

#pragma unroll 1
  for (int n = 0; n < nchunks; ++n) {
    const int st = n % STAGES;
    vmr[STAGES - 1] = issue_chunk(n + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t vm = vmr[0];
#pragma unroll
    for (int j = 0; j + 1 < STAGES; ++j) vmr[j] = vmr[j + 1];
    if (vm != 0) {  // warp-uniform: chunks of unused slots are passed over
      const uint32_t kt = my_s + st * C::STAGE_BYTES, vt = kt + TILE_BYTES;
      // ---- S^T = K_chunk . Q^T, two interleaved accumulator chains
      float sa[4] = {}, sb[4] = {};
#pragma unroll
      for (int kk = 0; kk < MT; kk += 2) {
        uint32_t a0, a1, a2, a3, e0, e1, e2, e3;
        ldmatrix_x4(kt + tile_off<D>(lane & 15, kk * 2 + (lane >> 4)), a0, a1, a2, a3);
        ldmatrix_x4(kt + tile_off<D>(lane & 15, (kk + 1) * 2 + (lane >> 4)), e0, e1, e2, e3);
        mma_bf16_16816(sa, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
        mma_bf16_16816(sb, e0, e1, e2, e3, qb[kk + 1][0], qb[kk + 1][1]);
      }
      // keys of this lane: lane/4 and lane/4 + 8; heads h0 = 2*(lane%4), h1 = h0 + 1
      const bool v0 = (vm >> (lane >> 2)) & 1u, v1 = (vm >> ((lane >> 2) + 8)) & 1u;
      const float x00 = v0 ? (sa[0] + sb[0]) * p.scale_log2 : -INFINITY;
      const float x01 = v0 ? (sa[1] + sb[1]) * p.scale_log2 : -INFINITY;
      const float x10 = v1 ? (sa[2] + sb[2]) * p.scale_log2 : -INFINITY;
      const float x11 = v1 ? (sa[3] + sb[3]) * p.scale_log2 : -INFINITY;
      float cm0 = fmaxf(x00, x10), cm1 = fmaxf(x01, x11);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        cm0 = fmaxf(cm0, __shfl_xor_sync(0xffffffffu, cm0, o));
        cm1 = fmaxf(cm1, __shfl_xor_sync(0xffffffffu, cm1, o));
      }
      // the max moves only by more than 8: every weight stays below 2^8
      const bool up0 = cm0 > m0 + 8.f, up1 = cm1 > m1 + 8.f;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float al0 = up0 ? exp2f(m0 - cm0) : 1.f, al1 = up1 ? exp2f(m1 - cm1) : 1.f;
        if (up0) m0 = cm0;
        if (up1) m1 = cm1;
        l0 *= al0;
        l1 *= al1;
        r0 *= al0;
        r1 *= al1;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          acc[mt][0] *= al0;
          acc[mt][1] *= al1;
          acc[mt][2] *= al0;
          acc[mt][3] *= al1;
        }
      }
      const float mu0 = m0 == -INFINITY ? 0.f : m0, mu1 = m1 == -INFINITY ? 0.f : m1;
      const float p00 = exp2f(x00 - mu0), p01 = exp2f(x01 - mu1);
      const float p10 = exp2f(x10 - mu0), p11 = exp2f(x11 - mu1);
      l0 += p00 + p10;
      l1 += p01 + p11;
      // P is rounded to bf16 for the product; O is divided by the sum of the rounded weights
      const uint32_t pk0 = pack_bf16x2(p00, p01), pk1 = pack_bf16x2(p10, p11);
      r0 += __uint_as_float(pk0 << 16) + __uint_as_float(pk1 << 16);
      r1 += __uint_as_float(pk0 & 0xFFFF0000u) + __uint_as_float(pk1 & 0xFFFF0000u);
      // ---- O^T += V^T . P^T
      const uint32_t pb0 = movmatrix_trans(pk0), pb1 = movmatrix_trans(pk1);
      const int vrow = (lane & 7) + ((lane >> 4) << 3), vseg_off = (lane >> 3) & 1;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t a0, a1, a2, a3;
        ldmatrix_x4_trans(vt + tile_off<D>(vrow, mt * 2 + vseg_off), a0, a1, a2, a3);
        mma_bf16_16816(acc[mt], a0, a1, a2, a3, pb0, pb1);
      }
    }
    __syncwarp();  // stage st is refilled by the next iteration's copies
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- the warp's state: sums over its lanes, O^T into its ring as [8][D]
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, o);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    r0 += __shfl_xor_sync(0xffffffffu, r0, o);
    r1 += __shfl_xor_sync(0xffffffffu, r1, o);
  }
  const int h0 = 2 * (lane % 4);
  float4* s_ml = reinterpret_cast<float4*>(smem + C::OFF_ML);
  if (lane < 4) {
    s_ml[warp * 8 + h0] = make_float4(m0, l0, r0, 0.f);
    s_ml[warp * 8 + h0 + 1] = make_float4(m1, l1, r1, 0.f);
  }
  float* wo = reinterpret_cast<float*>(my);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int d0 = mt * 16 + lane / 4;
    wo[h0 * D + d0] = acc[mt][0];
    wo[(h0 + 1) * D + d0] = acc[mt][1];
    wo[h0 * D + d0 + 8] = acc[mt][2];
    wo[(h0 + 1) * D + d0 + 8] = acc[mt][3];
  }
  __syncthreads();

  // ---- the block's state, sent to the blocks that finish the outputs: output e belongs to
  // block e % splits.  Every block of the cluster has started (the barrier's first phase).
  cg::cluster_group cluster = cg::this_cluster();
  float* s_co = reinterpret_cast<float*>(smem + C::OFF_CO);
  float4* s_cml = reinterpret_cast<float4*>(smem + C::OFF_CML);
  const int share = (8 * D + splits - 1) / splits;
  if (splits > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int e = threadIdx.x; e < p.G * D; e += WARPS * 32) {
    const int h = e / D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_ml[w * 8 + h].x);
    const float mu = M == -INFINITY ? 0.f : M;
    float o = 0.f, L = 0.f, R = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float4 ml = s_ml[w * 8 + h];
      const float f = exp2f(ml.x - mu);  // a warp without keys: 2^-inf = 0
      L = fmaf(ml.y, f, L);
      R = fmaf(ml.z, f, R);
      o = fmaf(reinterpret_cast<const float*>(smem + w * STAGES * C::STAGE_BYTES)[e], f, o);
    }
    if (splits == 1) {
      const long long head = row * p.Hq + g * p.G + h;
      p.O[head * D + e % D] = __bfloat16_as_ushort(__float2bfloat16_rn(R > 0.f ? o / R : 0.f));
      if (p.lse && e % D == 0) p.lse[head] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
    } else {
      cluster.map_shared_rank(s_co, e % splits)[rank * share + e / splits] = o;
      if (e % D < splits) cluster.map_shared_rank(s_cml, e % D)[rank * 8 + h] = make_float4(M, L, R, 0.f);
    }
  }
  if (splits == 1) return;  // block-uniform

  // ---- over the cluster: this block's outputs from every block's share, in order
  cluster.sync();
  for (int e = rank + threadIdx.x * splits; e < p.G * D; e += WARPS * 32 * splits) {
    const int h = e / D;
    float m[SAP_MAX_SPLITS], M = -INFINITY;
#pragma unroll
    for (int q = 0; q < SAP_MAX_SPLITS; ++q) {
      m[q] = q < splits ? s_cml[q * 8 + h].x : -INFINITY;
      M = fmaxf(M, m[q]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float o = 0.f, L = 0.f, R = 0.f;
#pragma unroll
    for (int q = 0; q < SAP_MAX_SPLITS; ++q) {
      if (q >= splits) continue;
      const float4 ml = s_cml[q * 8 + h];
      const float f = exp2f(m[q] - mu);
      L = fmaf(ml.y, f, L);
      R = fmaf(ml.z, f, R);
      o = fmaf(s_co[q * share + e / splits], f, o);
    }
    const long long head = row * p.Hq + g * p.G + h;
    p.O[head * D + e % D] = __bfloat16_as_ushort(__float2bfloat16_rn(R > 0.f ? o / R : 0.f));
    if (p.lse && e % D == 0) p.lse[head] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace dsa

namespace dsa_host {

template <int D, int WARPS>
static int sa_paged_launch_t(const dsa::SAPagedParams& p, long long groups, int splits, bool pdl, cudaStream_t stream) {
  constexpr int STAGES = 2;
  auto kern = dsa::sparse_attn_paged_kernel<D, WARPS, STAGES>;
  const int smem = dsa::SAPagedSmem<D, WARPS, STAGES>::BYTES;
  static DeviceFlag done;
  if (!done) {
    cudaError_t e_ = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e_ == cudaSuccess) e_ = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e_ != cudaSuccess) return cuda_fail(e_);
    done = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * splits));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (splits > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)splits;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, splits); e != cudaSuccess) return cuda_fail(e);
  return last_launch_status();
}

// While the (row, KV head) groups do not fill the SMs, blocks of 8 warps, one per SM, and the
// largest cluster that still gives every block an SM of its own and every warp a unit; past
// that, blocks of 4 warps without clusters.  Joining over a cluster costs about 2.5 us and a
// block's start as much again, so more and smaller pieces lose: 16 sequences of 2048 slots
// (64 groups) take 19.5 us as clusters of 2, 29 as clusters of 8; 64 sequences 48 us unsplit
// with 4 warps, 53 with 8, 58 as clusters of 2.
template <int D>
static int sa_paged_launch_d(const dsa::SAPagedParams& p, int batch, bool pdl, cudaStream_t stream) {
  const long long groups = (long long)batch * p.Hkv;
  const int sms = sm_count();
  if (groups > sms) return sa_paged_launch_t<D, 4>(p, groups, 1, pdl, stream);
  int splits = 1;
  while (splits < dsa::SAP_MAX_SPLITS && groups * splits * 2 <= sms && splits * 2 * 8 * 32 <= p.k) splits *= 2;
  return sa_paged_launch_t<D, 8>(p, groups, splits, pdl, stream);
}

int sparse_attn_paged_launch(const dsa::SAPagedParams& p, int batch, int d, bool pdl, cudaStream_t stream) {
  return d == 128 ? sa_paged_launch_d<128>(p, batch, pdl, stream) : sa_paged_launch_d<64>(p, batch, pdl, stream);
}

}  // namespace dsa_host

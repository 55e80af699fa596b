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
//
// Measured: 16 sequences, 2048 of 262144 positions each (67 MB), in 17.4 us, 17.8 launched
// eagerly: 2.6 us until the first copy starts (position, then its page, then its row), 10 us of
// streaming at 6.0 TB/s, 2 us to join the states; its 128 blocks leave 20 of the 148 SMs idle.  64
// sequences (270 MB) in 62 us, 54 where each has 8192 positions.  Halving the instructions of
// the gather changed nothing; more stages, or more warps per SM, neither.
#include <algorithm>
#include <cooperative_groups.h>
#include <type_traits>

#include "common.cuh"
#include "warp_mma.cuh"

namespace dsa {

__device__ __forceinline__ void cp_async_16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// An attention weight p >= 0 in two parts.  The heads of two weights as bf16 pairs, cut, not rounded:
// the rest is then never negative.
__device__ __forceinline__ uint32_t weight_heads(float p0, float p1) {
  return __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
}
// What the head leaves of p, at least the smallest bf16 (2^-133, nothing next to any weight) where
// p > 0: a rest of 0 would turn an infinity in V into NaN.
__device__ __forceinline__ float weight_rest(float p) {
  return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xFFFF0000u), fminf(p, 9.18354962e-41f));
}

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
  static constexpr int ROW = D * 2 + 16;              // padded: ldmatrix meets no bank twice
  static constexpr int STAGE_BYTES = 2 * 16 * ROW;    // K and V rows of a chunk
  static constexpr int TILE_BYTES = STAGE_BYTES / 2;
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int OFF_ML = RING;                    // [WARPS][8] float2: max, sum
  // what the cluster's blocks send to this one: the states of all of them, and their O of the
  // pieces (four dims of a head) that this block finishes
  static constexpr int OFF_CML = OFF_ML + WARPS * 8 * 8;             // [splits][8] float2
  static constexpr int OFF_CO = OFF_CML + SAP_MAX_SPLITS * 8 * 8;    // [splits][G D / 4 / splits] float4
  static constexpr int BYTES = OFF_CO + 8 * D * 4;
  static_assert(OFF_CO % 16 == 0, "float4");
  static_assert(STAGES * STAGE_BYTES >= 8 * D * 4, "a warp's O replaces its ring");
};

// SAME: both caches have the same page stride.
template <int D, int WARPS, int STAGES, bool SAME>
__global__ void __launch_bounds__(WARPS * 32) sparse_attn_paged_kernel(const SAPagedParams p, int splits) {
  namespace cg = cooperative_groups;
  using C = SAPagedSmem<D, WARPS, STAGES>;
  constexpr int MT = D / 16;
  pdl_wait();  // (loads below are plain: a read-only load may be moved above the wait)
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
  // the row's pages on their way to L2 while the positions load
  for (int i = threadIdx.x * 32; i < min(p.table_width, WARPS * 32 * 32 * 4); i += WARPS * 32 * 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(trow + i));

  const int len = max(p.lens[row], 0);
  uint32_t qb[MT][2];
  {
    const int head = lane / 4;
    const bool hv = head < p.G;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.Q + ((size_t)row * p.Hq + g * p.G + (hv ? head : 0)) * D);
#pragma unroll
    for (int kk = 0; kk < MT; ++kk) {
      qb[kk][0] = hv ? qrow[kk * 8 + (lane % 4)] : 0u;
      qb[kk][1] = hv ? qrow[kk * 8 + 4 + (lane % 4)] : 0u;
    }
  }

  // Slots are handled 32 at a time, a unit, one per lane: two chunks.  The chain position ->
  // page -> row is three dependent loads, so a unit's pages are looked up one unit ahead of its
  // copies and its positions two ahead.
  auto position = [&](int u) { return u < nunits && u * 32 + lane < p.k ? idx[u * 32 + lane] : -1; };
  // where a position's K and V rows start in the caches (bytes), or -1
  struct Slot {
    long long k, v;
  };
  // (two steps, so that nothing waits between a page's load and its use)
  auto page_of = [&](int s) {
    const int pg = s >> p.page_shift;
    return (unsigned)s < (unsigned)len && pg < p.table_width ? trow[pg] : -1;
  };
  auto slot_of = [&](int s, int page) -> Slot {
    if ((unsigned)page >= (unsigned)p.num_pages) return {-1, -1};
    const long long in = (long long)(s & ((1 << p.page_shift) - 1)) * kv_row;
    return {2 * (page * p.k_page_stride + in), SAME ? 0 : 2 * (page * p.v_page_stride + in)};
  };
  // starts the copies of a chunk, the lanes' slots from `first` on; returns its mask of valid
  // slots.  Eight lanes per row: each copy instruction moves 128-byte pieces of four rows.
  const uint32_t dst0 = my_s + (lane >> 3) * C::ROW + (lane & 7) * 16;
  const char* Kc = reinterpret_cast<const char*>(p.K + g * D) + (lane & 7) * 16;
  const char* Vc = reinterpret_cast<const char*>(p.V + g * D) + (lane & 7) * 16;
  auto issue = [&](int st, const Slot& mine, int first) -> uint32_t {
    const uint32_t vm = (__ballot_sync(0xffffffffu, mine.k >= 0) >> first) & 0xFFFFu;
    const uint32_t dst = dst0 + st * C::STAGE_BYTES;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = first + 4 * j + (lane >> 3);
      const long long ko = __shfl_sync(0xffffffffu, mine.k, r);
      const long long vo = SAME ? ko : __shfl_sync(0xffffffffu, mine.v, r);
      if (vm == 0xFFFFu) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          cp_async_16_all(dst + j * 4 * C::ROW + h * 128, Kc + ko + h * 128);
          cp_async_16_all(dst + C::TILE_BYTES + j * 4 * C::ROW + h * 128, Vc + vo + h * 128);
        }
      } else {  // slots that do not count are filled with zeros
        const bool valid = ko >= 0;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          cp_async_16(dst + j * 4 * C::ROW + h * 128, Kc + (valid ? ko : 0) + h * 128, valid);
          cp_async_16(dst + C::TILE_BYTES + j * 4 * C::ROW + h * 128, Vc + (valid ? vo : 0) + h * 128, valid);
        }
      }
    }
    cp_async_commit();
    return vm;
  };

  // ldmatrix addresses of this lane: K rows, and V rows transposed
  const uint32_t k_lane = my_s + (lane & 15) * C::ROW + (lane >> 4) * 16;
  const uint32_t v_lane = my_s + C::TILE_BYTES + ((lane & 7) + ((lane >> 4) << 3)) * C::ROW + ((lane >> 3) & 1) * 16;
  float acc[MT][4] = {};
  float m0 = -INFINITY, m1 = -INFINITY;  // running max (log2 domain) of heads h0, h1
  float l0 = 0.f, l1 = 0.f;              // this lane's share of the sums

  uint32_t vmr[STAGES];  // valid masks of the chunks in flight, the next one to use first
  int u_next = u0 + step;
  int s_cur = position(u0), s_next = position(u_next);
  int pg_cur = page_of(s_cur), pg_next = page_of(s_next);
  int s_far = position(u_next += step);
  Slot cs = slot_of(s_cur, pg_cur);
  auto issue_chunk = [&](int n) -> uint32_t {
    if (n >= nchunks) {
      cp_async_commit();
      return 0u;
    }
    if (n > 0 && n % 2 == 0) {  // the next unit
      cs = slot_of(s_next, pg_next);
      s_next = s_far;
      pg_next = page_of(s_next);
      s_far = position(u_next += step);
    }
    return issue(n % STAGES, cs, n % 2 * 16);
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
      // ---- S^T = K_chunk . Q^T, two interleaved accumulator chains
      float sa[4] = {}, sb[4] = {};
#pragma unroll
      for (int kk = 0; kk < MT; kk += 2) {
        uint32_t a0, a1, a2, a3, e0, e1, e2, e3;
        ldmatrix_x4(k_lane + st * C::STAGE_BYTES + kk * 32, a0, a1, a2, a3);
        ldmatrix_x4(k_lane + st * C::STAGE_BYTES + kk * 32 + 32, e0, e1, e2, e3);
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
      // ---- O^T += V^T . P^T, each weight as two bf16: its leading 8 bits, cut, and what that cuts
      // off, rounded, so 2^-16 of a weight is lost, not 2^-8.  Both are positive where the weight
      // is (see weight_rest), so that an infinity in V meets no other sign and no zero.  V's
      // fragments serve both products.
      const uint32_t hi0 = weight_heads(p00, p01), hi1 = weight_heads(p10, p11);
      const uint32_t lo0 = pack_bf16x2(weight_rest(p00), weight_rest(p01));
      const uint32_t lo1 = pack_bf16x2(weight_rest(p10), weight_rest(p11));
      const uint32_t b0 = movmatrix_trans(hi0), b1 = movmatrix_trans(hi1);
      const uint32_t c0 = movmatrix_trans(lo0), c1 = movmatrix_trans(lo1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t a0, a1, a2, a3;
        ldmatrix_x4_trans(v_lane + st * C::STAGE_BYTES + mt * 32, a0, a1, a2, a3);
        mma_bf16_16816(acc[mt], a0, a1, a2, a3, b0, b1);
        mma_bf16_16816(acc[mt], a0, a1, a2, a3, c0, c1);
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
  }
  const int h0 = 2 * (lane % 4);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  if (lane < 4) {
    s_ml[warp * 8 + h0] = make_float2(m0, l0);
    s_ml[warp * 8 + h0 + 1] = make_float2(m1, l1);
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

  // ---- the block's state, four dims of a head per thread, sent to the block that finishes them:
  // the G D / 4 pieces are dealt to the cluster's blocks (a power of two of them) in order.
  // Every block has started by then (the barrier's first phase).
  cg::cluster_group cluster = cg::this_cluster();
  float4* s_co = reinterpret_cast<float4*>(smem + C::OFF_CO);
  float2* s_cml = reinterpret_cast<float2*>(smem + C::OFF_CML);
  const int pieces = p.G * D / 4, share_log = 31 - __clz(pieces / splits);
  const long long head0 = row * p.Hq + g * p.G;
  // joins n states (max, sum) and O pieces, given by get(i, state, piece), in order
  auto join = [&](auto n, auto&& get, float& M, float& L, float4& o) {
    float2 ml[n.value];
    float4 x[n.value];
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < n.value; ++i) {
      get(i, ml[i], x[i]);
      M = fmaxf(M, ml[i].x);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    L = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < n.value; ++i) {
      const float f = exp2f(ml[i].x - mu);  // no keys: 2^-inf = 0
      L = fmaf(ml[i].y, f, L);
      o.x = fmaf(x[i].x, f, o.x);
      o.y = fmaf(x[i].y, f, o.y);
      o.z = fmaf(x[i].z, f, o.z);
      o.w = fmaf(x[i].w, f, o.w);
    }
  };
  auto finish = [&](int v, float M, float L, const float4& o) {
    const bool none = L == 0.f;  // a NaN sum is not an empty set
    const float inv = none ? 0.f : 1.f / L;
    const int h = v / (D / 4);
    *reinterpret_cast<uint2*>(p.O + head0 * D + v * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse && v % (D / 4) == 0) p.lse[head0 + h] = none ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
  };
  if (splits > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int v = threadIdx.x; v < pieces; v += WARPS * 32) {
    const int h = v / (D / 4);
    float M, L;
    float4 o;
    join(std::integral_constant<int, WARPS>(),
         [&](int w, float2& ml, float4& x) {
           ml = s_ml[w * 8 + h];
           x = reinterpret_cast<const float4*>(smem + w * STAGES * C::STAGE_BYTES)[v];
         },
         M, L, o);
    if (splits == 1) {
      finish(v, M, L, o);
    } else {
      const int owner = v >> share_log;
      cluster.map_shared_rank(s_co, owner)[(rank << share_log) + (v & ((1 << share_log) - 1))] = o;
      if (v % (D / 4) < splits) cluster.map_shared_rank(s_cml, v % (D / 4))[rank * 8 + h] = make_float2(M, L);
    }
  }
  if (splits == 1) return;  // block-uniform

  // ---- over the cluster: this block's pieces from every block's state, in order
  cluster.sync();
  for (int i = threadIdx.x; i < 1 << share_log; i += WARPS * 32) {
    const int v = (rank << share_log) + i, h = v / (D / 4);
    float M, L;
    float4 o;
    join(std::integral_constant<int, SAP_MAX_SPLITS>(),
         [&](int q, float2& ml, float4& x) {
           const bool in = q < splits;
           ml = in ? s_cml[q * 8 + h] : make_float2(-INFINITY, 0.f);
           x = in ? s_co[(q << share_log) + i] : make_float4(0.f, 0.f, 0.f, 0.f);
         },
         M, L, o);
    finish(v, M, L, o);
  }
}

}  // namespace dsa

namespace dsa_host {

template <int D, int WARPS, bool SAME>
static int sa_paged_launch_same(const dsa::SAPagedParams& p, long long groups, int splits, cudaStream_t stream) {
  constexpr int STAGES = 2;
  auto kern = dsa::sparse_attn_paged_kernel<D, WARPS, STAGES, SAME>;
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
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, splits); e != cudaSuccess) return cuda_fail(e);
  return last_launch_status();
}

template <int D, int WARPS>
static int sa_paged_launch_t(const dsa::SAPagedParams& p, long long groups, int splits, cudaStream_t stream) {
  return p.k_page_stride == p.v_page_stride ? sa_paged_launch_same<D, WARPS, true>(p, groups, splits, stream)
                                            : sa_paged_launch_same<D, WARPS, false>(p, groups, splits, stream);
}

// While the (row, KV head) groups do not fill the SMs: blocks of 8 warps, one per SM, in the
// largest cluster that still gives every block an SM of its own and every warp a unit, or of 4
// warps where those already give every unit its warp.  Past that, blocks of 4 warps, three per
// SM, without clusters.  Joining over a cluster costs about 1.5 us, so more and smaller pieces
// lose: 16 sequences of 2048 slots (64 groups) take 17.4 us as clusters of 2 blocks of 8 warps,
// 21.3 and 22.1 as clusters of 2 and 4 blocks of 4, 22.6 without clusters; 7 of 512 slots 6.2 us as
// clusters of 4 blocks of 4, 6.6 as clusters of 2 of 8.  Past one wave the two widths are close
// and neither always wins: 64 sequences of 2048 slots took 47 us with 4 warps and 50 with 8 when
// the rule was set, 62 and 52 later, from contexts of 262144 positions.
template <int D>
static int sa_paged_launch_d(const dsa::SAPagedParams& p, int batch, cudaStream_t stream) {
  const long long groups = (long long)batch * p.Hkv, sms = sm_count();
  if (groups > sms) return sa_paged_launch_t<D, 4>(p, groups, 1, stream);
  const int units = (p.k + 31) / 32;
  auto splits = [&](int warps) {
    int n = 1;
    while (n < dsa::SAP_MAX_SPLITS && groups * n * 2 <= sms && n * 2 * warps <= units) n *= 2;
    return n;
  };
  if (splits(4) * 4 >= units) return sa_paged_launch_t<D, 4>(p, groups, splits(4), stream);
  return sa_paged_launch_t<D, 8>(p, groups, splits(8), stream);
}

int sparse_attn_paged_launch(const dsa::SAPagedParams& p, int batch, int d, cudaStream_t stream) {
  return d == 128 ? sa_paged_launch_d<128>(p, batch, stream) : sa_paged_launch_d<64>(p, batch, stream);
}

}  // namespace dsa_host

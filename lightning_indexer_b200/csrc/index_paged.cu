// Indexer scores of one query row per sequence over a paged indexer-key cache (sm_100a).
//
//   scores[b, s] = sum_j w[b, j] * max(0, q_idx[b, j, :] . k_idx[position s of b]),  s < len_b
//
// Position s of sequence b is row s mod P of page table[b, s / P].  One query row reads every
// key of its sequence once: 2 d_I bytes and 2 H_I d_I operations per key, so with 64 heads
// the tensor cores are needed (64 operations per byte) and the keys' bytes set the floor.
//
// As in the contiguous indexer, 128 keys are the M side of a tcgen05 MMA and the heads its N
// side, so a thread of the epilogue owns one key and the ReLU, the weights and the head sum
// stay in its registers.  What differs:
//   - a tile of 128 keys is 128 / P pages (or part of one): the producer warp's lanes each
//     load one page piece by TMA, through a tensor map (dim, row, page); pages past the end
//     or outside the pool load as zeros through an out-of-range page coordinate;
//   - the tiles of all sequences form one list, cut evenly over the CTAs whatever the lengths
//     (each CTA sums the tile counts itself, there is no planning launch); a CTA walks its
//     piece of the list and reloads the query where it crosses into the next sequence.
//
// Measured: 16 sequences of 262144 positions, 1 GiB of keys, in 172 to 180 us (6.2 TB/s); 64
// ragged ones up to 16384 in 32.6 us, 33.5 launched eagerly (5.1 TB/s), of which 2.4 us pass before the first load
// (lengths, then the list, then the pages) and 1 after the last.
#include <algorithm>

#include "common.cuh"

namespace dsa {

// max(0, x), and NaN for NaN: a broken key or query must not score like an unrelated one.
__device__ __forceinline__ float relu(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

struct IndexPagedParams {
  const uint16_t* w;  // [batch, H_I]
  const int* lens;    // [batch]
  const int* table;   // [batch, table_width]
  int batch, table_width, page_shift, num_pages, max_len;
  float* scores;
  long long ld;
  int* cu_q;  // optional [batch + 1]: 0, 1, 2, ...
  int* cu_k;  // optional [batch + 1]: offsets of the (clamped) lengths
};

template <int H_I, int D_I>
struct IndexPagedCfg {
  static constexpr int N = H_I < 16 ? 16 : H_I;  // the heads past H_I are the next row's, unused
  static constexpr int PANEL = D_I >= 64 ? 64 : D_I;
  static constexpr int SWZ = PANEL * 2;
  static constexpr int NPANEL = D_I / PANEL;
  static constexpr int KSTEPS = PANEL / 16;
  static constexpr int A_BYTES = 128 * D_I * 2;
  static constexpr int B_BYTES = N * D_I * 2;
  static constexpr int A_STAGES = D_I == 128 ? 6 : D_I == 64 ? 12 : 16;  // 192 KB of keys in flight, or 128
  static constexpr int B_STAGES = 2, ACCS = 2;                           // accumulators in tensor memory
  static constexpr int TMEM_COLS = ACCS * N;
  static constexpr int PRODUCERS = 2;  // warps that load: warp 0 and the last one, every other tile each
  static constexpr int THREADS = 224;
  static_assert(A_STAGES % PRODUCERS == 0, "a producer's stages are its own");
  static constexpr int OFF_B = A_STAGES * A_BYTES;
  static constexpr int OFF_BAR = OFF_B + B_STAGES * B_BYTES;
  static constexpr int NUM_BARS = 2 * A_STAGES + 2 * B_STAGES + 2 * ACCS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
  static constexpr uint32_t IDESC = idesc_bf16_f32(128, N);
  static_assert(N <= 64 && SMEM_BYTES <= 232448, "limits");
};

// A CTA's walk over its piece of the tile list.
struct TileWalk {
  const IndexPagedParams& p;
  long long left;
  int b, t, len;
  __device__ __forceinline__ int length(int i) const {
    const long long cap = min((long long)p.max_len, (long long)p.table_width << p.page_shift);
    return (int)min((long long)max(p.lens[i], 0), cap);
  }
  __device__ __forceinline__ TileWalk(const IndexPagedParams& q, long long n, int b0, int t0) : p(q), left(n), b(b0), t(t0) {
    len = left > 0 ? length(b) : 0;
  }
  // tiles of the current sequence that belong to this CTA
  __device__ __forceinline__ int here() const { return (int)min(left, (long long)((len + 127) / 128 - t)); }
  __device__ __forceinline__ void next() {
    left -= here();
    t = 0;
    if (left <= 0) return;
    do {
      if (++b >= p.batch) {  // only if the lengths changed under the kernel
        left = 0;
        return;
      }
      len = length(b);
    } while (len == 0);
  }
};

template <int H_I, int D_I>
__global__ void __launch_bounds__(224, 1)
    index_paged_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_q,
                       const IndexPagedParams p) {
  using C = IndexPagedCfg<H_I, D_I>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::OFF_B;
  uint64_t* a_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* a_empty = a_full + C::A_STAGES;
  uint64_t* b_full = a_empty + C::A_STAGES;
  uint64_t* b_empty = b_full + C::B_STAGES;
  uint64_t* acc_full = b_empty + C::B_STAGES;
  uint64_t* acc_empty = acc_full + C::ACCS;
  uint64_t* mma_done = acc_empty + C::ACCS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  int* s_start = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);  // first sequence and tile of this CTA
  constexpr int WARPS = C::THREADS / 32;
  __shared__ long long warp_tiles[WARPS], warp_keys[WARPS];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::A_STAGES; ++i) mbar_init(&a_full[i], 1), mbar_init(&a_empty[i], 1);
    for (int i = 0; i < C::B_STAGES; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 1);
    for (int i = 0; i < C::ACCS; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 4);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // (loads below are plain: a read-only load may be moved above the wait)
  pdl_trigger();

  // the table on its way to L2 while the lengths load (the first 128 bytes per thread of the grid)
  if (const long long at = ((long long)blockIdx.x * C::THREADS + threadIdx.x) * 32; at < (long long)p.batch * p.table_width)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + at));

  // ---- the list of tiles: thread i sums a run of sequences, the block scans the sums
  long long first, count;
  {
    const TileWalk all(p, 0, 0, 0);
    const int per = (p.batch + C::THREADS - 1) / C::THREADS;
    const int lo = min((int)threadIdx.x * per, p.batch), hi = min(lo + per, p.batch);
    long long tiles = 0, keys = 0;
    for (int i = lo; i < hi; ++i) {
      const int n = all.length(i);
      tiles += (n + 127) / 128;
      keys += n;
    }
    long long xt = tiles, xk = keys;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, xt, o), c = __shfl_up_sync(0xffffffffu, xk, o);
      if (lane >= o) xt += a, xk += c;
    }
    if (lane == 31) warp_tiles[warp] = xt, warp_keys[warp] = xk;
    __syncthreads();
    long long bt = xt - tiles, bk = xk - keys, total = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) bt += warp_tiles[i], bk += warp_keys[i];
      total += warp_tiles[i];
    }
    first = total * blockIdx.x / gridDim.x;
    count = total * (blockIdx.x + 1) / gridDim.x - first;
    if (count > 0 && first >= bt && first < bt + tiles) {
      int i = lo;
      long long at = bt;
      for (;; ++i) {
        const int nt = (all.length(i) + 127) / 128;
        if (first < at + nt) break;
        at += nt;
      }
      s_start[0] = i;
      s_start[1] = (int)(first - at);
    }
    if (p.cu_k && blockIdx.x == 0) {
      for (int i = lo; i < hi; ++i) {
        p.cu_q[i] = i;
        p.cu_k[i] = (int)bk;
        bk += all.length(i);
      }
      if (hi == p.batch && lo < hi) p.cu_q[p.batch] = p.batch, p.cu_k[p.batch] = (int)bk;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int b0 = count > 0 ? s_start[0] : 0, t0 = count > 0 ? s_start[1] : 0;

  if (warp == 0 || warp == WARPS - 1) {
    // ------------------------------------------------------------ TMA producers (whole warps)
    // A page piece costs a warp about 50 ns to issue, 16 pieces to a tile of 16-row pages: two
    // warps take the tiles by turns.
    const int producer = warp == 0 ? 0 : 1;
    const int box_rows = min(1 << p.page_shift, 128);
    const int pieces = 128 / box_rows;  // of a tile
    const int piece = lane / C::NPANEL, panel = lane % C::NPANEL;
    const bool mine = piece < pieces;
    int as = 0, bs = 0;
    uint32_t aph = 0, bph = 0;
    bool ok = true;
    for (TileWalk w(p, count, b0, t0); w.left > 0 && ok; w.next()) {
      const int* row = p.table + (long long)w.b * p.table_width;
      // The pages of 32 consecutive pieces of the sequence, one per lane, loaded a batch ahead
      // and looked at only when used: a lookup per tile put a memory latency into every tile.
      auto pages_from = [&](int q) {
        const long long s = (long long)(q + lane) * box_rows;
        return s < w.len ? row[s >> p.page_shift] : -1;
      };
      int q0 = w.t * pieces, ids = pages_from(q0), ids_next = pages_from(q0 + 32);
      if (producer == 0 && lane == 0) {
        if ((ok = mbar_wait(&b_empty[bs], bph ^ 1, abort_flag, 41))) {
          mbar_arrive_expect_tx(&b_full[bs], C::B_BYTES);
          for (int pn = 0; pn < C::NPANEL; ++pn)
            tma_load_2d(sB + bs * C::B_BYTES + pn * C::N * C::SWZ, &tmap_q, &b_full[bs], pn * C::PANEL, w.b * H_I);
        }
      }
      if (!(ok = __shfl_sync(0xffffffffu, ok, 0))) break;
      if (++bs == C::B_STAGES) { bs = 0; bph ^= 1; }
      const int end = w.t + w.here();
      for (int t = w.t; t < end; ++t) {
        if (t * pieces == q0 + 32) {
          q0 += 32;
          ids = ids_next;
          ids_next = pages_from(q0 + 32);
        }
        if (as % C::PRODUCERS != producer) {  // the other warp's stage
          if (++as == C::A_STAGES) { as = 0; aph ^= 1; }
          continue;
        }
        // a page outside the pool loads zeros: num_pages is past the map's last one
        const int id = __shfl_sync(0xffffffffu, ids, (t * pieces - q0 + piece) & 31);
        const int cur = (unsigned)id < (unsigned)p.num_pages ? id : p.num_pages;
        if (lane == 0) {
          if ((ok = mbar_wait(&a_empty[as], aph ^ 1, abort_flag, 42))) mbar_arrive_expect_tx(&a_full[as], C::A_BYTES);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (mine)
          tma_load_3d(sA + as * C::A_BYTES + panel * 128 * C::SWZ + piece * box_rows * C::SWZ, &tmap_k, &a_full[as],
                      panel * C::PANEL, (t * 128 + piece * box_rows) & ((1 << p.page_shift) - 1), cur);
        __syncwarp();
        if (++as == C::A_STAGES) { as = 0; aph ^= 1; }
      }
    }
    if (!ok && lane == 0) {
      // drain: let every load this warp issued land before the CTA can exit
      for (int i = producer; i < C::A_STAGES; i += C::PRODUCERS) {
        const uint64_t t1 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&a_full[i]), aph ^ (i >= as ? 1u : 0u)) && globaltimer_ns() - t1 < 200000000ull) {
        }
      }
      for (int i = 0; i < C::B_STAGES && producer == 0; ++i) {
        const uint64_t t1 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&b_full[i]), bph ^ (i >= bs ? 1u : 0u)) && globaltimer_ns() - t1 < 200000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int as = 0, bs = 0, ab = 0;
      uint32_t aph = 0, bph = 0, abph = 0;
      bool ok = true;
      for (TileWalk w(p, count, b0, t0); w.left > 0 && ok; w.next()) {
        if (!(ok = mbar_wait(&b_full[bs], bph, abort_flag, 43))) break;
        const uint32_t b_base = smem_u32(sB + bs * C::B_BYTES);
        for (int n = w.here(); n > 0; --n) {
          if (!(ok = mbar_wait(&acc_empty[ab], abph ^ 1, abort_flag, 44))) break;
          if (!(ok = mbar_wait(&a_full[as], aph, abort_flag, 45))) break;
          tc_fence_after();
          const uint32_t a_base = smem_u32(sA + as * C::A_BYTES);
          const uint32_t d_tmem = tmem_base + ab * C::N;
#pragma unroll
          for (int pn = 0; pn < C::NPANEL; ++pn)
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS; ++kk)
              umma_bf16(d_tmem, smem_desc_kmajor(a_base + pn * 128 * C::SWZ + kk * 32, C::SWZ),
                        smem_desc_kmajor(b_base + pn * C::N * C::SWZ + kk * 32, C::SWZ), C::IDESC, (pn | kk) != 0);
          umma_commit(&a_empty[as]);
          umma_commit(&acc_full[ab]);
          if (++as == C::A_STAGES) { as = 0; aph ^= 1; }
          if (++ab == C::ACCS) { ab = 0; abph ^= 1; }
        }
        if (!ok) break;
        umma_commit(&b_empty[bs]);
        if (++bs == C::B_STAGES) { bs = 0; bph ^= 1; }
      }
      // every MMA this thread issued, before tensor memory can be released
      umma_commit(mma_done);
      const uint64_t t1 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(mma_done), 0) && globaltimer_ns() - t1 < 200000000ull) {
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int lane_grp = warp % 4;
    const uint32_t lane_off = (uint32_t)(lane_grp * 32) << 16;
    int ab = 0;
    uint32_t abph = 0;
    bool ok = true;
    for (TileWalk w(p, count, b0, t0); w.left > 0 && ok; w.next()) {
      float wr[H_I];
#pragma unroll
      for (int h = 0; h < H_I; h += 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p.w + (long long)w.b * H_I + h);
        wr[h] = __uint_as_float(v.x << 16);
        wr[h + 1] = __uint_as_float(v.x & 0xffff0000u);
        wr[h + 2] = __uint_as_float(v.y << 16);
        wr[h + 3] = __uint_as_float(v.y & 0xffff0000u);
      }
      const int* row = p.table + (long long)w.b * p.table_width;
      float* out = p.scores + (long long)w.b * p.ld;
      const int end = w.t + w.here();
      auto page_at = [&](int s) { return s < w.len ? row[s >> p.page_shift] : -1; };
      int id_next = page_at(w.t * 128 + lane_grp * 32 + lane);
      for (int t = w.t; t < end; ++t) {
        const int s = t * 128 + lane_grp * 32 + lane;
        const int id = id_next;
        id_next = page_at(s + 128);  // a tile ahead of its use
        if (!(ok = mbar_wait(&acc_full[ab], abph, abort_flag, 46))) break;
        __syncwarp();  // the loads below are warp-wide
        tc_fence_after();
        const uint32_t tbase = tmem_base + lane_off + ab * C::N;
        float acc = 0.f;
#pragma unroll
        for (int h0 = 0; h0 < H_I; h0 += 16) {
          float v[16];
          tmem_ld_x16_sync(tbase + h0, v);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (h0 + q < H_I) acc = fmaf(wr[h0 + q < H_I ? h0 + q : 0], relu(v[q]), acc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ab]);
        if (s < w.len) out[s] = (unsigned)id < (unsigned)p.num_pages ? acc : -INFINITY;
        if (++ab == C::ACCS) { ab = 0; abph ^= 1; }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::TMEM_COLS);
}

}  // namespace dsa

namespace dsa_host {

template <int H_I, int D_I>
static int index_paged_launch_t(const void* q_idx, const void* k_cache, long long page_stride,
                                const dsa::IndexPagedParams& p, cudaStream_t stream) {
  using C = dsa::IndexPagedCfg<H_I, D_I>;
  auto kern = dsa::index_paged_kernel<H_I, D_I>;
  static DeviceFlag attr_done;
  const int smem = std::max(C::SMEM_BYTES, 120 * 1024);  // one CTA per SM
  if (!attr_done) {
    if (const cudaError_t e_ = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); e_ != cudaSuccess) return cuda_fail(e_);
    attr_done = true;
  }
  CUtensorMap tk, tq;
  const uint64_t P = 1ull << p.page_shift;
  const uint64_t dims[3] = {(uint64_t)D_I, P, (uint64_t)p.num_pages};
  const uint64_t strides[2] = {(uint64_t)D_I * 2, (uint64_t)page_stride * 2};
  const uint32_t box[3] = {(uint32_t)C::PANEL, (uint32_t)std::min<uint64_t>(P, 128), 1};
  int st = make_tmap_bf16_3d(&tk, k_cache, dims, strides, box, C::SWZ);
  if (st != DSA_OK) return st;
  st = make_tmap_bf16_2d(&tq, q_idx, (uint64_t)p.batch * H_I, D_I, (uint64_t)D_I * 2, C::N, C::PANEL, C::SWZ);
  if (st != DSA_OK) return st;
  const long long tiles = (long long)p.batch * ((p.max_len + 127) / 128);
  const long long grid = std::max<long long>(1, std::min<long long>(tiles, sm_count()));
  return launch_pdl(true, kern, dim3((unsigned)grid), dim3(C::THREADS), (size_t)smem, stream, tk, tq, p);
}

int index_paged_launch(const void* q_idx, const void* k_cache, long long page_stride, const dsa::IndexPagedParams& p,
                       int H_I, int d_I, cudaStream_t stream) {
  if (H_I == 64 && d_I == 128) return index_paged_launch_t<64, 128>(q_idx, k_cache, page_stride, p, stream);
  if (H_I == 32 && d_I == 128) return index_paged_launch_t<32, 128>(q_idx, k_cache, page_stride, p, stream);
  if (H_I == 16 && d_I == 128) return index_paged_launch_t<16, 128>(q_idx, k_cache, page_stride, p, stream);
  if (H_I == 8 && d_I == 64) return index_paged_launch_t<8, 64>(q_idx, k_cache, page_stride, p, stream);
  if (H_I == 4 && d_I == 32) return index_paged_launch_t<4, 32>(q_idx, k_cache, page_stride, p, stream);
  return DSA_ERR_UNSUPPORTED;
}

}  // namespace dsa_host

// A few rows times a weight matrix: one read of the weights is all the time
// there is.  The operands change places: 128 rows of the weights are the MMA's
// M, the tokens (16, 32, 48 or 64, padded by the TMA with zeros) its N.  A tile's K
// is shared out over a cluster of up to 8 CTAs, so that a few dozen tiles keep
// every SM loading; each CTA streams its share through a ring of TMA stages,
// and the partial sums meet through distributed shared memory, added in the
// order of the ranks.  For the gated form a tile holds rows of the gate's weights
// and as many of the up projection's for the same channels.  A tile may have fewer
// than 128 rows (a multiple of 8: what the MMA reads beyond them reaches no result),
// so that the tiles come out even over the SMs (few_shape).
#include "few.cuh"

namespace tpk {
namespace product {
namespace {

constexpr int kFewThreads = 128;

template <int kTok>
struct FewSmem {
  static constexpr int kStages = kTok == 16 ? 6 : kTok == 32 ? 5 : 4;   // two CTAs per SM
  uint8_t a[kStages][kBoxBytes];
  uint8_t b[kStages][kTok * 128];
  uint64_t full[kStages], empty[kStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
};
template <int kTok>
constexpr size_t kFewBytes = sizeof(FewSmem<kTok>) + 1024;

struct FewParams {
  int32_t N, O, k_iters;     // tokens, results per token (of one of the two, gated), stages of K
  int32_t rows;              // channels of a tile
  int32_t act;
  const float* bias;
  const __nv_bfloat16* residual;
  int64_t ld_res;
  __nv_bfloat16* y;
  int64_t ld_y;
  int32_t* err;
};

struct FewMaps {
  CUtensorMap w, w2, x;
};

template <int kTok, bool kGated>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ FewMaps maps, const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Sm = FewSmem<kTok>;
  constexpr int kS = Sm::kStages;
  Sm& S = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(S.a[0]);   // [kTok][128], once the stages have been read
  static_assert(kTok * 512 <= kS * kBoxBytes, "partial sums");
  constexpr int kCols = kTok <= 32 ? 32 : 64;     // TMEM columns
  const int warp = threadIdx.x >> 5;
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int tile = blockIdx.x / ranks;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.k_iters) * rank / ranks);
  const int nk = static_cast<int>(static_cast<int64_t>(p.k_iters) * (rank + 1) / ranks) - k0;
  volatile int* abort_flag = &S.abort_flag;

  if (kGated) ptx::dependents_launch();
  auto weights = [&](int st, int k) {
    ptx::mbar_arrive_expect_tx(&S.full[st], (kGated ? 2 : 1) * p.rows * 128 + kTok * 128);
    ptx::tma_load_2d(S.a[st], &maps.w, &S.full[st], (k0 + k) * 64, tile * p.rows);
    if (kGated) ptx::tma_load_2d(S.a[st] + p.rows * 128, &maps.w2, &S.full[st], (k0 + k) * 64, tile * p.rows);
  };
  const int first = nk < kS ? nk : kS;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    ptx::mbar_init(&S.done, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
    // the first weights are on their way while the CTA sets itself up; they wait
    // for no earlier kernel
    for (int k = 0; k < first; ++k) weights(k, k);
  }
  if (warp == 2) {
    ptx::tmem_alloc(&S.tmem_base, kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  if (warp == 0) {
    if (threadIdx.x == 0) {
      ptx::dependency_wait();
      for (int k = 0; k < first; ++k) ptx::tma_load_2d(S.b[k], &maps.x, &S.full[k], (k0 + k) * 64, 0);
      int issued = first;
      for (int k = kS; k < nk; ++k, ++issued) {
        const int st = k % kS;
        if (!ptx::mbar_wait(&S.empty[st], (k / kS - 1) & 1, abort_flag, kWaitLimitNs)) break;
        weights(st, k);
        ptx::tma_load_2d(S.b[st], &maps.x, &S.full[st], (k0 + k) * 64, 0);
      }
      // nothing is left in flight, whatever became of the products
      for (int k = issued > kS ? issued - kS : 0; k < issued; ++k) ptx::mbar_drain(&S.full[k % kS], (k / kS) & 1);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, kTok, false, false);
      for (int k = 0; k < nk; ++k) {
        const int st = k % kS;
        if (!ptx::mbar_wait(&S.full[st], (k / kS) & 1, abort_flag, kWaitLimitNs)) break;
        ptx::tc_fence_after();
        const uint64_t ad = ptx::sw128_desc(ptx::smem_addr(S.a[st]), 16, 1024);
        const uint64_t bd = ptx::sw128_desc(ptx::smem_addr(S.b[st]), 16, 1024);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          ptx::mma_ss(tmem, ptx::desc_add(ad, q * 32), ptx::desc_add(bd, q * 32), idesc, (k > 0 || q > 0) ? 1u : 0u);
        ptx::mma_commit(&S.empty[st]);
      }
      ptx::mma_commit(&S.done);
    }
  }
  __syncwarp();
  ptx::dependency_wait();
  // Every product issued has been done, and the producer's last loads have landed: the
  // stages are free.  One answer for all threads: a warp reads TMEM as a whole.
  const bool ok = __syncthreads_and(ptx::mbar_drain(&S.done, 0));
  ptx::tc_fence_after();
  // every thread's row of the accumulator (a result's channel) to shared memory, channels side by side
  if (ok) {
#pragma unroll
    for (int c = 0; c < kTok; c += 16) {
      uint32_t r[16];
      ptx::tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, r);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) red[(c + e) * 128 + threadIdx.x] = __uint_as_float(r[e]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // every CTA's partial sums are there
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
  if ((!ok || S.abort_flag) && threadIdx.x == 0 && p.err) *p.err = TPK_E_TIMEOUT;

  // this CTA's share of the channels, four at a time
  const int quads = (p.rows / 4 + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
  for (int i = threadIdx.x; i < p.N * quads; i += kFewThreads) {
    const int t = i / quads, at = (static_cast<int>(rank) * quads + i % quads) * 4;
    const int o = tile * p.rows + at;
    if (at >= p.rows || o >= p.O) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
    for (uint32_t k = 0; k < ranks; ++k) {
      const float4 d = ptx::lds128_cluster(red + t * 128 + at, k);
      v.x += d.x; v.y += d.y; v.z += d.z; v.w += d.w;
      if (kGated) {
        const float4 e = ptx::lds128_cluster(red + t * 128 + p.rows + at, k);
        u.x += e.x; u.y += e.y; u.z += e.z; u.w += e.w;
      }
    }
    if (!kGated && p.bias) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + o));
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    with_act(p.act, [&](auto k) {
      constexpr int kAct = decltype(k)::value;
      ptx::unf2(act_2<kAct>(ptx::f2(v.x, v.y)), v.x, v.y);
      ptx::unf2(act_2<kAct>(ptx::f2(v.z, v.w)), v.z, v.w);
    });
    if (kGated) {
      v.x *= u.x; v.y *= u.y; v.z *= u.z; v.w *= u.w;
    } else if (p.residual) {
      const uint2 q = *reinterpret_cast<const uint2*>(p.residual + t * p.ld_res + o);
      v.x += lo16(q.x); v.y += hi16(q.x); v.z += lo16(q.y); v.w += hi16(q.y);
    }
    *reinterpret_cast<uint2*>(p.y + t * p.ld_y + o) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  }
  ptx::cluster_sync();   // nobody reads a CTA that has gone
}

// Channels per tile and CTAs that share a tile's K (each with two stages or more):
// the pair that leaves the busiest SM the least to read, weights and tokens, of
// those whose clusters all run together (a second round of clusters cost one token,
// 2,048 to 4,096, 11.0 us against 8.5); among equals the one with most CTAs.  More
// channels than that: full tiles, one CTA each.  Two CTAs run per SM; of the clusters
// of 4 and 8 all but two are at home at once (74 and 36 on 152 SMs; the runtime's
// occupancy query counts one CTA per SM for kernels that use tensor memory).  (40
// tokens, width 4,096, 12,288 gated channels: 48 channels a tile 36 us, 64 39; one
// token, width 8,192 to 2,048, 128 channels: 8 CTAs 12 us, 4 about 14, 1 27.)
struct FewShape {
  int rows, ranks;
  int64_t tiles;
};
FewShape few_shape(int64_t O, bool gated, int tok, int k_iters) {
  const int most_rows = gated ? 64 : 128, sms = num_sms();
  FewShape best{most_rows, 1, (O + most_rows - 1) / most_rows};
  double least = 0.0;
  for (int ranks = 1; ranks <= 8 && (ranks == 1 || k_iters >= 2 * ranks); ranks *= 2)
    for (int rows = most_rows; rows >= most_rows / 2; rows -= 8) {
      const int64_t tiles = (O + rows - 1) / rows, ctas = tiles * ranks;
      if (tiles > 2 * sms / ranks - (ranks > 2 ? 2 : 0)) continue;
      // (one CTA alone on its SM leaves it idle at its ends)
      const double read = static_cast<double>((ctas + sms - 1) / sms * ((gated ? 2 : 1) * rows + tok)) / ranks *
                          (ctas > sms ? 1.0 : 1.15);
      if (least == 0.0 || read < least || (read == least && ctas > best.tiles * best.ranks)) {
        least = read;
        best = FewShape{rows, ranks, tiles};
      }
    }
  return best;
}

struct FewConfig {   // a launch of clusters of `ranks` CTAs
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  FewConfig(int64_t tiles, int ranks, size_t smem, bool after, cudaStream_t s) {
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * ranks));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = after ? 2 : 1;
  }
};

template <int kTok, bool kGated>
int few_launch(const Mat& x, const Mat& w, const Mat& w2, FewParams& p, bool after, cudaStream_t s) {
  constexpr auto kern = few_kernel<kTok, kGated>;
  static PerContext<int> rec;
  int st = guarded([&] { return set_smem_once(rec, kern, kFewBytes<kTok>); });
  if (st != TPK_OK) return st;
  const FewShape shape = few_shape(p.O, kGated, kTok, p.k_iters);
  p.rows = shape.rows;
  FewMaps m;
  st = map_of(&m.w, w, shape.rows);
  if (st == TPK_OK) st = map_of(&m.x, x, kTok);
  if (st == TPK_OK && kGated) st = map_of(&m.w2, w2, shape.rows);
  if (st != TPK_OK) return st;
  FewConfig c(shape.tiles, shape.ranks, kFewBytes<kTok>, after, s);
  return launched(cudaLaunchKernelEx(&c.cfg, kern, m, p));
}

template <bool kGated>
int few_dispatch(const Mat& x, const Mat& w, const Mat& w2, FewParams& p, bool after, cudaStream_t s) {
  p.N = static_cast<int32_t>(x.rows);
  p.O = static_cast<int32_t>(w.rows);
  p.k_iters = static_cast<int32_t>((w.cols + 63) / 64);
  const int tok = (p.N + 15) / 16 * 16;
  return tok == 16   ? few_launch<16, kGated>(x, w, w2, p, after, s)
         : tok == 32 ? few_launch<32, kGated>(x, w, w2, p, after, s)
         : tok == 48 ? few_launch<48, kGated>(x, w, w2, p, after, s)
                     : few_launch<64, kGated>(x, w, w2, p, after, s);
}

}  // namespace

int few_linear(const Mat& x, const Mat& w, const float* bias, int act, const Mat& residual, const Mat& y, bool after,
               int32_t* err, cudaStream_t s) {
  FewParams p{};
  p.act = act;
  p.bias = bias;
  p.residual = static_cast<const __nv_bfloat16*>(residual.p);
  p.ld_res = residual.ld;
  p.y = static_cast<__nv_bfloat16*>(const_cast<void*>(y.p));
  p.ld_y = y.ld;
  p.err = err;
  return few_dispatch<false>(x, w, w, p, after, s);
}

int few_gate(const Mat& x, const Mat& w_gate, const Mat& w_up, int act, const Mat& a, int32_t* err, cudaStream_t s) {
  FewParams p{};
  p.act = act;
  p.y = static_cast<__nv_bfloat16*>(const_cast<void*>(a.p));
  p.ld_y = a.ld;
  p.err = err;
  return few_dispatch<true>(x, w_gate, w_up, p, false, s);
}

}  // namespace product
}  // namespace tpk

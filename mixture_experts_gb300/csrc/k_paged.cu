// Paged decode attention: choice of the kernel's form, and the join of the
// segments that block borders cut.
#include "../../include/coli_moe.h"
#include "paged_launch.cuh"

namespace coli {
namespace paged {
namespace {

// Block (c, y) joins the segment that starts in block c of the main kernel and
// ends in a later one: its partial means o with weight sums l at maxima m, in the order
// of the blocks, o = sum o_k l_k 2^(m_k - m) / sum l_k 2^(m_k - m), four at a time and a mean
// throughout (sums could overflow where the result does not). A group of registers is one 16 x 8 tile of
// O^T. With gridDim.y = 1 a warp takes whole groups; otherwise block y takes
// group y and its warps share the partials. Latency bound: 6 to 8 us by itself, of
// which the launch lies under the main kernel (one context of 500009 tokens: 38
// partials a segment, 7.4 us; 32 ragged contexts: 2 a segment, 6.0 us).
template <int DP, int NT, bool F32, bool IN_ORDER, bool EXT>
__global__ void __launch_bounds__(256) k_join(const Params p) {
  constexpr int kGroups = DP / 16 * NT, kRegs = kGroups * 4;
  constexpr int kPart = kRegs * 32 + 16 * NT;
  __shared__ float s_o[8][4][32], s_ml[8][4][4];
  const int lane = lane_id(), w = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  const PagedArgs& a = p.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 sp = p.span[blockIdx.x];
  if (sp.w == 0) return;
  const bool shared = gridDim.y > 1;
  const int step = shared ? 8 : 1, D = a.c.head_dim;
  for (int gr = shared ? blockIdx.y : w; gr < kGroups; gr += shared ? kGroups : 8) {
    const int i = gr / NT, nt = gr - i * NT;
    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kBatch = 4;
    for (int k = shared ? w : 0; k < sp.w; k += step * kBatch) {
      float pm[kBatch][2], pl[kBatch][2], po[kBatch][4];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int kk = k + e * step;
        const bool in = kk < sp.w;
        const float* src =
            p.part + static_cast<size_t>(2 * (blockIdx.x + kk) + (kk == 0 ? sp.z : 0)) * kPart;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          pm[e][c] = in ? src[kRegs * 32 + nt * 8 + 2 * t + c] : -FLT_MAX;
          pl[e][c] = in ? src[kRegs * 32 + 8 * NT + nt * 8 + 2 * t + c] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) po[e][c] = in ? src[gr * 128 + c * 32 + lane] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = m[c];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) top = fmaxf(top, pm[e][c]);
        const float f = l[c] * ex2(m[c] - top);
        float sum = f;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          pl[e][c] *= ex2(pm[e][c] - top);
          sum += pl[e][c];
        }
        const float by = sum == 0.f ? 0.f : reciprocal(sum);
        o[c] *= f * by;
        o[c + 2] *= f * by;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          o[c] = fmaf(po[e][c], pl[e][c] * by, o[c]);
          o[c + 2] = fmaf(po[e][c + 2], pl[e][c] * by, o[c + 2]);
        }
        m[c] = top;
        l[c] = sum;
      }
    }
    if (shared) {
#pragma unroll
      for (int c = 0; c < 4; ++c) s_o[w][c][lane] = o[c];
      if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) s_ml[w][t][c] = m[c], s_ml[w][t][2 + c] = l[c];
      }
      __syncthreads();
      if (w != 0) return;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[c] = -FLT_MAX;
        for (int k = 0; k < 8; ++k) m[c] = fmaxf(m[c], s_ml[k][t][c]);
        l[c] = o[c] = o[c + 2] = 0.f;
        for (int k = 0; k < 8; ++k) l[c] += s_ml[k][t][2 + c] * ex2(s_ml[k][t][c] - m[c]);
        const float by = l[c] == 0.f ? 0.f : reciprocal(l[c]);
        for (int k = 0; k < 8; ++k) {
          const float f = s_ml[k][t][2 + c] * ex2(s_ml[k][t][c] - m[c]) * by;
          o[c] = fmaf(s_o[k][c][lane], f, o[c]);
          o[c + 2] = fmaf(s_o[k][c + 2][lane], f, o[c + 2]);
        }
      }
    }
    const int b = sp.x, h = sp.y / p.blocks, row0 = (sp.y - h * p.blocks) * 8 * NT;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = row0 + nt * 8 + 2 * t + c;
      if (r >= p.group) continue;
      store_out<IN_ORDER, F32, EXT>(a, row_at<EXT>(a, p.group, b, h, r, a.out_stride, D), i, g,
                               l[c] == 0.f ? 0.f : o[c], l[c] == 0.f ? 0.f : o[c + 2]);
      if (a.lse != nullptr && i == 0 && g == 0) store_lse<EXT>(a, p.group, b, h, r, m[c], l[c]);
    }
  }
}

// The join is launched so that its blocks may be placed while the main kernel
// drains; they wait for its end (griddepcontrol.wait) before they read.
template <int DP, int NT, bool F32, bool IN_ORDER, bool EXT>
cudaError_t launch_join(const Params& p, int grid, int ys, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, ys);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_join<DP, NT, F32, IN_ORDER, EXT>, p);
}

struct Form {
  int dp, nt, blocks, per_sm, warps;
  size_t part;  // floats of a partial slot
};

template <int FMT, int DP, int NT>
void fill(Form* f) {
  using C = Cfg<FMT, DP, NT>;
  f->per_sm = C::kPerSm;
  f->warps = C::kWarps;
  f->part = C::kPart;
}

template <int FMT>
void fill_format(Form* f) {
  if constexpr (FMT != DT_F32) {
    if (f->nt == 2)
      return f->dp == 64    ? fill<FMT, 64, 2>(f)
             : f->dp == 128 ? fill<FMT, 128, 2>(f)
                            : fill<FMT, 256, 2>(f);
  }
  if (f->dp == 64) return fill<FMT, 64, 1>(f);
  if (f->dp == 128) return fill<FMT, 128, 1>(f);
  fill<FMT, 256, 1>(f);
}

Form form_of(const KvView& c, int n_q_heads) {
  Form f{};
  const int group = n_q_heads / c.n_heads;
  f.dp = c.head_dim <= 64 ? 64 : (c.head_dim <= 128 ? 128 : 256);
  f.nt = group <= 8 || c.dtype == DT_F32 ? 1 : 2;
  f.blocks = (group + 8 * f.nt - 1) / (8 * f.nt);
  switch (c.dtype) {
    case DT_F32: fill_format<DT_F32>(&f); break;
    case DT_BF16: fill_format<DT_BF16>(&f); break;
    case DT_MXFP8: fill_format<DT_MXFP8>(&f); break;
    default: fill_format<DT_MXFP4>(&f);
  }
  return f;
}

template <bool F32, bool IN_ORDER, bool EXT>
cudaError_t launch_joins(const Params& p, const Form& f, int grid, int ys, cudaStream_t st) {
  if constexpr (!F32) {
    if (f.nt == 2)
      return f.dp == 64    ? launch_join<64, 2, F32, IN_ORDER, EXT>(p, grid, ys, st)
             : f.dp == 128 ? launch_join<128, 2, F32, IN_ORDER, EXT>(p, grid, ys, st)
                           : launch_join<256, 2, F32, IN_ORDER, EXT>(p, grid, ys, st);
  }
  if (f.dp == 64) return launch_join<64, 1, F32, IN_ORDER, EXT>(p, grid, ys, st);
  if (f.dp == 128) return launch_join<128, 1, F32, IN_ORDER, EXT>(p, grid, ys, st);
  return launch_join<256, 1, F32, IN_ORDER, EXT>(p, grid, ys, st);
}

template <bool EXT>
cudaError_t run(const Params& p, const Form& f, int grid, int64_t segments, cudaStream_t st) {
  cudaError_t e;
  switch (p.a.c.dtype) {
    case DT_F32: e = (EXT ? launch_f32_ext : launch_f32)(p, f.dp, f.nt, grid, st); break;
    case DT_BF16: e = (EXT ? launch_bf16_ext : launch_bf16)(p, f.dp, f.nt, grid, st); break;
    case DT_MXFP8: e = (EXT ? launch_mxfp8_ext : launch_mxfp8)(p, f.dp, f.nt, grid, st); break;
    default: e = (EXT ? launch_mxfp4_ext : launch_mxfp4)(p, f.dp, f.nt, grid, st); break;
  }
  if (e != cudaSuccess || p.direct) return e;
  // long segments (many partials each): the warps of a block share a group
  const int groups = f.dp / 16 * f.nt;
  const int ys = segments * 4 < grid ? groups : 1;
  switch (p.a.c.dtype) {
    case DT_F32: return launch_joins<true, false, EXT>(p, f, grid, ys, st);
    case DT_BF16: return launch_joins<false, true, EXT>(p, f, grid, ys, st);
    default: return launch_joins<false, false, EXT>(p, f, grid, ys, st);
  }
}

}  // namespace
}  // namespace paged

int sm_count() {
  static int n[128] = {};
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 152;
  if (n[dev] == 0 &&
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    n[dev] = v;
  return n[dev] ? n[dev] : 152;
}

size_t paged_scratch_bytes(const KvView& c, int B, int n_q_heads) {
  const paged::Form f = paged::form_of(c, n_q_heads);
  const size_t blocks = static_cast<size_t>(sm_count()) * f.per_sm;
  return blocks * (2 * f.part * sizeof(float) + sizeof(int4));
}

bool paged_direct(const KvView& c, int max_pages) {
  return static_cast<int64_t>(max_pages) * c.page_size <= COLI_PAGED_DIRECT_TOKENS;
}

cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t st) {
  using namespace paged;
  const Form f = form_of(a.c, a.n_q_heads);
  const int most = sm_count() * f.per_sm;
  Params p{};
  p.a = a;
  p.group = a.n_q_heads / a.c.n_heads;
  p.blocks = f.blocks;
  p.part = a.scratch;
  p.span = reinterpret_cast<int4*>(a.scratch + 2 * f.part * most);
  // no more blocks than pieces of one tile a warp
  const int64_t segments = static_cast<int64_t>(a.B) * a.c.n_heads * f.blocks;
  const int64_t tiles = static_cast<int64_t>(a.max_pages) * (a.c.page_size / kTile);
  const int64_t pieces = (segments * (tiles + 8) + f.warps - 1) / f.warps;
  // One block a segment, nothing cut, where the block table holds 1024 tokens at most (which
  // callers know, and need no scratch then), or 2048 and the segments fill the GPU. Direct
  // against cut and joined, us, heads of 128, at 100 / 300 / 500 / 1000 tokens:
  //   bf16  B 1, 32/8 heads   4.7-7.0   5.8-6.9   6.8-7.0   9.4-7.2
  //         B 1, 8/1          4.9-5.9   6.2-6.7   6.9-6.7   9.5-6.8
  //         B 4, 32/8         4.9-8.6   6.1-8.5   6.9-9.5   9.5-10.1
  //         B 16, 32/8        5.2-8.7   6.6-10.8  9.9-14.0  14.8-18.6
  //   MXFP8 B 1, 32/8         6.5-9.7   9.9-9.9   11.1-9.9  17.2-10.1
  //         B 4, 32/8         6.7-12.1  10.1-12.2 11.7-12.7 18.5-13.2
  //         B 16, 32/8        7.5-10.6  11.3-11.6 12.7-14.1 20.2-22.5
  //   MXFP4 B 1, 64/4         7.8-9.8   11.0-10.0 14.2-10.3 21.8-10.6
  //   f32   B 1, 16/8         7.2-9.6   12.7-9.6  16.2-9.6  27.4-9.9
  // and bf16 at 2000, B 128: 104-117. So it is the faster form for short contexts and for
  // full batches; a few sequences of 500 to 1000 tokens would be faster cut (up to 2.8
  // times in fp32), which needs scratch that such a call may leave out.
  p.direct = paged_direct(a.c, a.max_pages) ||
             (static_cast<int64_t>(a.max_pages) * a.c.page_size <= 2 * COLI_PAGED_DIRECT_TOKENS &&
              segments >= most);
  // A caller that has the scratch in any case: too few segments for the GPU are cut from the
  // lengths on where the table above has it faster.
  const int64_t tokens = static_cast<int64_t>(a.max_pages) * a.c.page_size;
  if (a.ext && a.may_cut && segments < most &&
      tokens >= (a.c.dtype == DT_F32 ? 192 : a.c.dtype == DT_BF16 ? 512 : 320))
    p.direct = 0;
  const int grid = p.direct ? static_cast<int>(segments)
                            : (pieces < most ? static_cast<int>(pieces) : most);
  return a.ext ? run<true>(p, f, grid, segments, st) : run<false>(p, f, grid, segments, st);
}

}  // namespace coli

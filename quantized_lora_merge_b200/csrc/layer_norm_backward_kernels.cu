// Gradients of the layer norm over the rows of a tokens x n activation. With
// xh_j = (x_j - m) rstd and g_j = dy_j w_j, m and rstd of the forward:
//
//   dx_j = rstd (g_j - mean g - xh_j mean(g xh)),
//   dw_j = sum_t dy_tj xh_tj, db_j = sum_t dy_tj
//
// Bound by memory: 14 operations an element against 6 to 12 bytes. dx and both
// sums over rows come from one read of x and dy; sums and products are fp32, dx is
// rounded once. How rows are spread over threads, and the ring that brings them
// in, is layer_norm_rows.cuh.
#include <type_traits>

#include "layer_norm_rows.cuh"

namespace intlora {

namespace {

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Every thread keeps the sums of its columns of dy xh and dy in registers over
// all its rows; at the end the block's teams are joined in shared memory, in a
// fixed order, and written once, as row blockIdx.x of partial
// ([blocks][2][n]). Up to kHoldV chunks a thread, xh and g stay in registers
// between the row sums and dx; above, the ring is read a second time.
template <int TX, int TY, typename F>
__global__ void __launch_bounds__(kBlock, 1)
    layer_norm_backward_kernel(const __grid_constant__ LayerNormBackwardJob j, const __grid_constant__ RowShape r,
                               float* partial) {
  char* ring = smem();
  __shared__ float scratch[2][2 * 32];
  constexpr bool kHold = F::V <= kHoldV;
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  const bool idle = team >= r.teams;           // threads behind the last whole team: touch nothing
  float* weight = reinterpret_cast<float*>(ring + r.params);
  const uint32_t mine = static_cast<uint32_t>(min(team, r.teams - 1) * r.stages * r.stage_bytes);
  const Columns<F> c(t, n);
  const int64_t step = static_cast<int64_t>(gridDim.x) * r.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const int64_t ahead = step * (r.stages - 1);
  const int64_t x_step = step * j.ld_x * elem_bytes(j.x_type), dy_step = step * j.ld_dy * elem_bytes(j.dy_type);
  const int64_t dx_step = step * j.ld_dx * elem_bytes(j.dx_type);
  const char* next_x = static_cast<const char*>(row_ptr(j.x, row, j.ld_x, j.x_type));
  const char* next_dy = static_cast<const char*>(row_ptr(j.dy, row, j.ld_dy, j.dy_type));
  const char* here_x = next_x;
  const char* here_dy = next_dy;
  char* dx = j.dx != nullptr ? static_cast<char*>(row_ptr(j.dx, row, j.ld_dx, j.dx_type)) : nullptr;
  const auto fetch = [&](int slot, int64_t which) {
    if (which < j.tokens && !idle) {
      const uint32_t stage = mine + slot * r.stage_bytes;
      fetch_row<kBytes<TX>, F>(stage, next_x, j.x, n, t, T);
      fetch_row<kBytes<TY>, F>(stage + r.second, next_dy, j.dy, n, t, T);
    }
    copy_commit();
    next_x += x_step;
    next_dy += dy_step;
  };
  const int width = max(T, F::L) * F::V * kChunk;          // columns of a team's slots
  clear_tails(ring, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.x_type) / 16 * 16, r.second);
  clear_tails(ring + r.second, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.dy_type) / 16 * 16,
              r.stage_bytes - r.second);
  if (!F::VEC) __syncthreads();                   // copies write there too, later
  for (int s = 0; s + 1 < r.stages; ++s) fetch(s, row + s * step);
  const auto stat = [&](const float* p, int64_t at) { return at < j.tokens && !idle ? p[at] : 0.0f; };
  float mean = stat(j.mean, row), rstd = stat(j.rstd, row);
  stage_params<F::VEC>(weight, j.weight, j.param_type, n, width, 1.0f);
  __syncthreads();
  F2 dw[2 * F::V], db[2 * F::V];
#pragma unroll
  for (int i = 0; i < 2 * F::V; ++i) dw[i] = db[i] = f2(0.0f);
  if (T <= 32 || !idle) {
    int slot = 0, flip = 0;
    for (int64_t base = row - team; base < j.tokens; base += step) {
      const bool live = row < j.tokens && !idle;
      fetch(slot == 0 ? r.stages - 1 : slot - 1, row + ahead);
      const F2 m = f2(-mean), scale = f2(rstd);
      mean = stat(j.mean, row + step);         // a row ahead, like the ring
      rstd = stat(j.rstd, row + step);
      copy_wait(r.stages - 1);
      arrive_sync<F::VEC>(T, team);
      const uint32_t sx = mine + slot * r.stage_bytes + (F::VEC ? 0 : granule_shift(here_x));
      const uint32_t sy = mine + slot * r.stage_bytes + r.second + (F::VEC ? 0 : granule_shift(here_dy));
      F2 xh[kHold ? 2 * F::V : 2], g[kHold ? 2 * F::V : 2], s0 = f2(0.0f), s1 = f2(0.0f);
      // xh, dy and w of chunk k
      const auto load = [&](int k, F2* px, F2* py, F2* pw) {
        read_chunk<TX, F>(sx, j.x_type, c, k, px[0], px[1]);
        read_chunk<TY, F>(sy, j.dy_type, c, k, py[0], py[1]);
        param_chunk<F>(r.params, c, k, pw[0], pw[1]);
        // columns past n: xh is zero like x and dy; -mean rstd may be beyond fp32,
        // and NaN in the row's sums (up to 3 % of the time; a second sum for such
        // rows alone spills, and takes more)
        if constexpr (F::VEC) {
          const F2 mk = c.has(k, 0) ? m : f2(0.0f);
          px[0] = (px[0] + mk) * scale;
          px[1] = (px[1] + mk) * scale;
        } else {
          const float m1 = split(m).x;
          px[0] = (px[0] + f2(c.has(k, 0) ? m1 : 0.0f, c.has(k, 1) ? m1 : 0.0f)) * scale;
          px[1] = (px[1] + f2(c.has(k, 2) ? m1 : 0.0f, c.has(k, 3) ? m1 : 0.0f)) * scale;
        }
      };
      if (live) {
#pragma unroll
        for (int k = 0; k < F::V; ++k) {
          F2* px = xh + (kHold ? 2 * k : 0);
          F2* pg = g + (kHold ? 2 * k : 0);
          F2 dy[2], w[2];
          load(k, px, dy, w);
          pg[0] = dy[0] * w[0];
          pg[1] = dy[1] * w[1];
          s0 = s0 + (pg[0] + pg[1]);
          s1 = fma2(pg[0], px[0], fma2(pg[1], px[1], s1));
          dw[2 * k] = fma2(dy[0], px[0], dw[2 * k]);
          dw[2 * k + 1] = fma2(dy[1], px[1], dw[2 * k + 1]);
          db[2 * k] = db[2 * k] + dy[0];
          db[2 * k + 1] = db[2 * k + 1] + dy[1];
        }
      }
      if (j.dx != nullptr) {                   // uniform over the grid
        float s[2] = {both(s0), both(s1)};
        team_sum<2>(s, T, team, scratch[flip]);
        flip ^= 1;
        const F2 c1 = f2(-s[0] * inv_n), c2 = f2(-s[1] * inv_n);
        if (live) {
          const auto finish = [&](auto td) {
            constexpr int TD = decltype(td)::value;
            if constexpr (kHold) {
#pragma unroll
              for (int i = 0; i < 2 * F::V; ++i) xh[i] = scale * fma2(xh[i], c2, g[i] + c1);
              write_typed<TD, F>(dx, j.dx_type, c, xh);
            } else {
#pragma unroll
              for (int k = 0; k < F::V; ++k) {
                F2 dy[2], w[2];
                load(k, xh, dy, w);
                write_chunk<TD, F, false>(dx, j.dx_type, c, k, scale * fma2(xh[0], c2, fma2(dy[0], w[0], c1)),
                                               scale * fma2(xh[1], c2, fma2(dy[1], w[1], c1)));
              }
            }
          };
          if (j.dx_type == kF32) finish(std::integral_constant<int, kF32>{});
          else finish(std::integral_constant<int, TX == kF32 ? kAny16 : TX>{});
        }
      }
      arrive_sync<F::VEC>(T, team);               // the slot is free for the next copy
      slot = slot + 1 == r.stages ? 0 : slot + 1;
      row += step;
      here_x += x_step;
      here_dy += dy_step;
      if (dx != nullptr) dx += dx_step;
    }
  }
  if (partial == nullptr) return;
  if (r.teams == 1 && T >= 32) {               // nothing to join
    if (idle) return;
    char* out = reinterpret_cast<char*>(partial + static_cast<int64_t>(blockIdx.x) * 2 * n);
    write_typed<kF32, F>(out, kF32, c, dw);
    write_typed<kF32, F>(out + static_cast<size_t>(n) * 4, kF32, c, db);
    return;
  }
  copy_wait(0);
  __syncthreads();                             // the ring becomes the teams' sums: [team][2][width]
  float* sums = reinterpret_cast<float*>(ring);
  int rows = r.teams;
  if (T < 32) {                                // teams of one warp first
    rows = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < 2 * F::V; ++i)
      for (int o = T; o < 32; o <<= 1) {
        F2 p, q;
        p.v = __shfl_xor_sync(0xffffffffu, dw[i].v, o);
        q.v = __shfl_xor_sync(0xffffffffu, db[i].v, o);
        dw[i] = dw[i] + p;
        db[i] = db[i] + q;
      }
  }
  if (T >= 32 ? !idle : (threadIdx.x & 31) < T) {
    float2* to = reinterpret_cast<float2*>(sums + static_cast<size_t>(T >= 32 ? team : threadIdx.x >> 5) * 2 * width) + t;
    const int lanes = max(T, F::L);
#pragma unroll
    for (int i = 0; i < 2 * F::V; ++i) {
      to[i * lanes] = split(dw[i]);
      to[width / 2 + i * lanes] = split(db[i]);
    }
  }
  __syncthreads();
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * n;
  for (int col = threadIdx.x; col < 2 * n; col += blockDim.x) {
    const int cc = col < n ? col : col - n;
    // lanes, pair and half that hold column cc
    const int in = cc % (F::V * F::kCols), group = cc / (F::V * F::kCols);
    const int elem = F::VEC ? in / F::kCols * kChunk + in % kChunk : in / 32;
    const int lane = F::VEC ? in % F::kCols / kChunk : in % 32;
    const int at = ((elem >> 1) * max(T, F::L) + group * F::L + lane) * 2 + (elem & 1) + (col < n ? 0 : width);
    float s = sums[at];
    for (int k = 1; k < rows; ++k) s += sums[static_cast<size_t>(k) * 2 * width + at];
    out[col] = s;
  }
}

// dx of rows too wide for registers.
__global__ void __launch_bounds__(kWideThreads)
    layer_norm_backward_wide_kernel(const __grid_constant__ LayerNormBackwardJob j) {
  __shared__ float scratch[2][2 * 32];
  int flip = 0;
  for (int64_t row = blockIdx.x; row < j.tokens; row += gridDim.x) {
    const void* x = row_ptr(j.x, row, j.ld_x, j.x_type);
    const void* dy = row_ptr(j.dy, row, j.ld_dy, j.dy_type);
    const float mean = j.mean[row], rstd = j.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float w = j.weight != nullptr ? load_elem(j.weight, c, j.param_type) : 1.0f;
      const float g = load_elem(dy, c, j.dy_type) * w;
      s[0] += g;
      s[1] = fmaf(g, (load_elem(x, c, j.x_type) - mean) * rstd, s[1]);
    }
    team_sum<2>(s, kWideThreads, 0, scratch[flip]);
    flip ^= 1;
    const float c1 = s[0] / static_cast<float>(j.n), c2 = s[1] / static_cast<float>(j.n);
    void* dx = row_ptr(j.dx, row, j.ld_dx, j.dx_type);
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float w = j.weight != nullptr ? load_elem(j.weight, c, j.param_type) : 1.0f;
      const float xh = (load_elem(x, c, j.x_type) - mean) * rstd;
      store_elem(dx, c, j.dx_type, rstd * (fmaf(load_elem(dy, c, j.dy_type), w, -c1) - xh * c2));
    }
  }
}

// Column sums of dy xh and dy for wide rows: a thread owns a column over the
// rows of its split.
__global__ void __launch_bounds__(kColThreads)
    layer_norm_columns_kernel(const __grid_constant__ LayerNormBackwardJob j, float* partial) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (c >= j.n) return;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < j.tokens; row += gridDim.y) {
    const float dy = load_elem(row_ptr(j.dy, row, j.ld_dy, j.dy_type), c, j.dy_type);
    const float x = load_elem(row_ptr(j.x, row, j.ld_x, j.x_type), c, j.x_type);
    dw = fmaf(dy, (x - j.mean[row]) * j.rstd[row], dw);
    db += dy;
  }
  float* out = partial + static_cast<int64_t>(blockIdx.y) * 2 * j.n;
  out[c] = dw;
  out[j.n + c] = db;
}

// dweight and dbias from the blocks' partial sums, added in block order.
__global__ void __launch_bounds__(32 * kReduceWarps)
    layer_norm_reduce_kernel(const float* partial, int64_t blocks, int64_t n, float* dweight, float* dbias,
                             int accumulate) {
  __shared__ float part[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  wait_for_previous();
  if (c < 2 * n) {
#pragma unroll 8
    for (int64_t p = warp; p < blocks; p += kReduceWarps) s += partial[p * 2 * n + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * n) return;
  s = part[0][lane];
#pragma unroll
  for (int k = 1; k < kReduceWarps; ++k) s += part[k][lane];
  float* out = c < n ? dweight : dbias;
  if (out == nullptr) return;
  const int64_t at = c < n ? c : c - n;
  out[at] = accumulate ? out[at] + s : s;
}

template <int TX, int TY, typename F>
cudaError_t launch_bwd(const LayerNormBackwardJob& j, const RowShape& r, unsigned grid, size_t smem, float* partial,
                       cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(layer_norm_backward_kernel<TX, TY, F>), &done);
  if (e != cudaSuccess) return e;
  layer_norm_backward_kernel<TX, TY, F><<<grid, r.threads(), smem, s>>>(j, r, partial);
  return counted(cudaGetLastError());
}

template <int TX, int TY>
cudaError_t bwd_by_v(const LayerNormBackwardJob& j, const RowShape& r, bool vec, unsigned grid, size_t smem,
                     float* partial, cudaStream_t s) {
  if (r.L == 16) {
    switch (r.V) {
      case 2: return launch_bwd<TX, TY, Form<2, true, 16>>(j, r, grid, smem, partial, s);
      case 3: return launch_bwd<TX, TY, Form<3, true, 16>>(j, r, grid, smem, partial, s);
      case 4: return launch_bwd<TX, TY, Form<4, true, 16>>(j, r, grid, smem, partial, s);
      case 5: return launch_bwd<TX, TY, Form<5, true, 16>>(j, r, grid, smem, partial, s);
      case 6: return launch_bwd<TX, TY, Form<6, true, 16>>(j, r, grid, smem, partial, s);
      case 8: return launch_bwd<TX, TY, Form<8, true, 16>>(j, r, grid, smem, partial, s);
    }
    return cudaErrorInvalidConfiguration;
  }
  switch (vec ? r.V : -r.V) {
    case 1: return launch_bwd<TX, TY, Form<1, true>>(j, r, grid, smem, partial, s);
    case 2: return launch_bwd<TX, TY, Form<2, true>>(j, r, grid, smem, partial, s);
    case 3: return launch_bwd<TX, TY, Form<3, true>>(j, r, grid, smem, partial, s);
    case 4: return launch_bwd<TX, TY, Form<4, true>>(j, r, grid, smem, partial, s);
    case 5: return launch_bwd<TX, TY, Form<5, true>>(j, r, grid, smem, partial, s);
    case 6: return launch_bwd<TX, TY, Form<6, true>>(j, r, grid, smem, partial, s);
    case 8: return launch_bwd<TX, TY, Form<8, true>>(j, r, grid, smem, partial, s);
    case -1: return launch_bwd<TX, TY, Form<1, false>>(j, r, grid, smem, partial, s);
    case -2: return launch_bwd<TX, TY, Form<2, false>>(j, r, grid, smem, partial, s);
    case -4: return launch_bwd<TX, TY, Form<4, false>>(j, r, grid, smem, partial, s);
    case -6: return launch_bwd<TX, TY, Form<6, false>>(j, r, grid, smem, partial, s);
    case -8: return launch_bwd<TX, TY, Form<8, false>>(j, r, grid, smem, partial, s);
  }
  return cudaErrorInvalidConfiguration;
}
cudaError_t bwd_by_type(const LayerNormBackwardJob& j, const RowShape& r, bool vec, unsigned grid, size_t smem,
                        float* partial, cudaStream_t s) {
  const bool x32 = j.x_type == kF32, y32 = j.dy_type == kF32;
  // bf16 has kernels of its own, where dx is bf16 or fp32 too; the other pairs
  // with 16-bit types select between the conversions
  if (j.x_type == kBf16 && j.dx_type != kF16) {
    if (j.dy_type == kBf16) return bwd_by_v<kBf16, kBf16>(j, r, vec, grid, smem, partial, s);
    if (y32) return bwd_by_v<kBf16, kF32>(j, r, vec, grid, smem, partial, s);
  }
  if (x32 && y32) return bwd_by_v<kF32, kF32>(j, r, vec, grid, smem, partial, s);
  if (x32) return bwd_by_v<kF32, kAny16>(j, r, vec, grid, smem, partial, s);
  if (y32) return bwd_by_v<kAny16, kF32>(j, r, vec, grid, smem, partial, s);
  return bwd_by_v<kAny16, kAny16>(j, r, vec, grid, smem, partial, s);
}

}  // namespace

namespace {
// The number of partial sums depends on tokens and n alone, so that the
// workspace does: as many blocks as SMs, if there are rows for them. Rows too
// wide for the ring (two fp32 tensors, any alignment) go to the wide kernels.
struct BackwardSums {
  bool wide = false;
  int64_t blocks = 0;
};
BackwardSums backward_sums(int64_t tokens, int64_t n) {
  BackwardSums b;
  RowShape r;
  b.wide = !row_shape(RowWant{tokens, n, false, kBwdMaxV, kF32, kF32, 1}, &r) ||
           !row_shape(RowWant{tokens, n, true, kBwdMaxV, kF32, kF32, 1}, &r);
  const int64_t strips = (n + kColThreads - 1) / kColThreads;
  b.blocks = b.wide ? std::min<int64_t>(std::max<int64_t>(1, kSms * 8 / strips), std::max<int64_t>(1, tokens / 8))
                    : std::max<int64_t>(1, std::min<int64_t>(kSms, tokens));
  return b;
}
}  // namespace

size_t layer_norm_backward_ws(int64_t tokens, int64_t n) {
  const BackwardSums b = backward_sums(tokens, n);
  return (static_cast<size_t>(b.blocks) * 2 * static_cast<size_t>(n) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardJob& j, void* ws, cudaStream_t s) {
  const BackwardSums b = backward_sums(j.tokens, j.n);
  const bool sums = j.dweight != nullptr || j.dbias != nullptr;
  float* partial = sums ? static_cast<float*>(ws) : nullptr;
  if (b.wide) {
    if (sums) {                                // first: dx may take the place of dy or x
      const dim3 grid(static_cast<unsigned>((j.n + kColThreads - 1) / kColThreads), static_cast<unsigned>(b.blocks));
      layer_norm_columns_kernel<<<grid, kColThreads, 0, s>>>(j, partial);
      const cudaError_t e = counted(cudaGetLastError());
      if (e != cudaSuccess) return e;
    }
    if (j.dx != nullptr && j.tokens > 0) {
      layer_norm_backward_wide_kernel<<<grid_of(j.tokens, 1 << 20), kWideThreads, 0, s>>>(j);
      const cudaError_t e = counted(cudaGetLastError());
      if (e != cudaSuccess) return e;
    }
  } else if (j.dx != nullptr || sums) {
    const bool vec = rows_aligned(j.x, j.ld_x, j.n, j.x_type) && rows_aligned(j.dy, j.ld_dy, j.n, j.dy_type) &&
                     (j.dx == nullptr || rows_aligned(j.dx, j.ld_dx, j.n, j.dx_type)) &&
                     reinterpret_cast<uintptr_t>(j.weight) % 16 == 0;
    RowShape r;
    // single elements take more registers: V = 8 spills (3000 x 5003: 65 us, V = 6 58)
    if (!row_shape(RowWant{j.tokens, j.n, vec, vec ? kBwdMaxV : 6, j.x_type, j.dy_type, 1}, &r) &&
        !row_shape(RowWant{j.tokens, j.n, vec, kBwdMaxV, j.x_type, j.dy_type, 1}, &r))
      return cudaErrorInvalidConfiguration;
    // the joined sums take the place of ring and parameters
    const size_t join = static_cast<size_t>(r.T >= 32 ? r.teams : r.threads() / 32) * 2 * slot_columns(r) * sizeof(float);
    const size_t smem = std::max(static_cast<size_t>(r.params) + static_cast<size_t>(slot_columns(r)) * sizeof(float), join);
    const cudaError_t e = bwd_by_type(j, r, vec, static_cast<unsigned>(b.blocks), smem, partial, s);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  return counted(launch_after(layer_norm_reduce_kernel, static_cast<unsigned>((2 * j.n + 31) / 32), 32 * kReduceWarps, 0, s,
                              partial, b.blocks, j.n, j.dweight, j.dbias, j.accumulate));
}

}  // namespace intlora

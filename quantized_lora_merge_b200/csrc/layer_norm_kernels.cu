// Layer norm over the rows of a tokens x n activation.
//
//   m = mean_j x_j, v = mean_j (x_j - m)^2, rstd = (v + eps)^-1/2,
//   y_j = (x_j - m) rstd w_j + b_j
//
// Bound by memory: 8 operations an element against 4 to 8 bytes. Both sums run
// over registers, two passes over the values and one over memory; statistics and
// products are fp32, y is rounded once. How rows are spread over threads, and the
// ring that brings them in, is layer_norm_rows.cuh.
#include "layer_norm_rows.cuh"

namespace intlora {

namespace {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Whether a row's spread may be nothing but the error of its mean: a mean of
// `steps` roundings is off by up to steps x 2^-24 of it, and the row of equal
// values c, whose spread is zero, shows |c - mean| as its spread. Rows in registers
// (17 additions in a thread, 5 across a warp, 32 across warps, the factor 1 / n):
// standard deviations below 2^-18 of the mean.
constexpr float kRowSteps = 64.0f;
__device__ __forceinline__ bool spread_in_doubt(float mean, float var, float steps) {
  const float off = steps * 0x1p-24f * mean;
  return mean != 0.0f && var <= off * off;
}

// Mean and variance of a row in doubt, formed again about a corrected mean. What
// a row of equal values has left over its mean is exact and has few bits, so the
// sums of that are exact, and so are their quotients by n (not by a rounded 1 / n):
// it ends at its value and at the variance zero. Teams of one warp come here
// together; those not in doubt keep what they have. `less` is what the row less
// its old mean is to be reduced by.
struct Moments {
  float mean, var, less;
};
__device__ __noinline__ Moments settle_row(const void* row, int type, int64_t count, float n, int t, int T, int team,
                                           float* scratch, bool doubt, float mean, float var) {
  float s[1] = {0.0f}, s2[2] = {0.0f, 0.0f};
  for (int64_t c = t; c < count; c += T) s[0] += load_elem(row, c, type) - mean;
  team_sum<1>(s, T, team, scratch);
  const float better = mean + s[0] / n;
  for (int64_t c = t; c < count; c += T) {
    const float v = load_elem(row, c, type) - better;
    s2[0] += v;
    s2[1] = fmaf(v, v, s2[1]);
  }
  team_sum<2>(s2, T, team, scratch + 32);
  if (!doubt) return Moments{mean, var, 0.0f};
  const float rest = s2[0] / n;                // what the better mean has lost to rounding
  return Moments{better + rest, fmaxf(fmaf(-rest, rest, s2[1] / n), 0.0f), (better - mean) + rest};
}

// A row in doubt, from its elements on: x is still what it was, in shared memory
// or, where the row is not written yet, in memory. Parameters: fp32 in shared
// memory, or those of the job (weight == nullptr). For such rows alone, at the row's
// end and out of line, where little is live. us: 8192 x 4096 bf16 28.6, fp32 36.3 (in
// line behind the sums 32.1 and 36.7, all rows corrected there 30.1 and 43.3,
// nothing corrected 28.6 and 36.1); what is left is the test of every row: 16384 x
// 320 fp16 6.96 (6.72 without), 30000 x 40 fp32 7.4 (7.0).
__device__ __noinline__ void redo_row(const LayerNormJob& j, const void* x, int64_t row, int count, const float* weight,
                                      const float* bias, int t, int T, int team, float* scratch, bool doubt, float mean,
                                      float var) {
  team_sync(T, team);                          // what the team wrote comes before what it writes here
  const Moments m = settle_row(x, j.x_type, count, static_cast<float>(j.n), t, T, team, scratch, doubt, mean, var);
  if (doubt) {
    const float rstd = rsqrtf(m.var + j.eps);
    if (t == 0) {
      if (j.mean != nullptr) j.mean[row] = m.mean;
      if (j.rstd != nullptr) j.rstd[row] = rstd;
    }
    void* y = row_ptr(j.y, row, j.ld_y, j.y_type);
    for (int c = t; c < count; c += T) {
      float o = ((load_elem(x, c, j.x_type) - mean) - m.less) * rstd;
      if (weight != nullptr) {
        o = fmaf(o, weight[c], bias[c]);
      } else {
        if (j.weight != nullptr) o *= load_elem(j.weight, c, j.param_type);
        if (j.bias != nullptr) o += load_elem(j.bias, c, j.param_type);
      }
      store_elem(y, c, j.y_type, o);
    }
  }
  team_sync(T, team);                          // the row's place may be taken
}

// Mean, variance and rstd of a row held in registers; x becomes x - mean. scratch: five
// parts of 32, of which the last three are redo_row's, so that no barrier stands
// between the reads of one sum and the writes of the next.
constexpr int kScratch = 5 * 32;
template <typename F>
__device__ __forceinline__ void row_stats(F2 (&x)[2 * F::V], const Columns<F>& c, float inv_n, float eps, int T,
                                          int team, float* scratch, float* mean_out, float* var_out, float* rstd_out) {
  F2 a = x[0], b = x[1];
#pragma unroll
  for (int k = 1; k < F::V; ++k) {
    a = a + x[2 * k];
    b = b + x[2 * k + 1];
  }
  float s[1] = {both(a + b)};
  team_sum<1>(s, T, team, scratch);
  const float mean = s[0] * inv_n;
  a = b = f2(0.0f);
  if (!F::VEC && c.full()) {
    const F2 m = f2(-mean);
#pragma unroll
    for (int k = 0; k < F::V; ++k) {
      x[2 * k] = x[2 * k] + m;
      x[2 * k + 1] = x[2 * k + 1] + m;
      a = fma2(x[2 * k], x[2 * k], a);
      b = fma2(x[2 * k + 1], x[2 * k + 1], b);
    }
  } else {
#pragma unroll
    for (int k = 0; k < F::V; ++k) {              // zeros behind n stay zeros
      F2 mp, mq;
      if (F::VEC) {
        mp = mq = f2(c.has(k, 0) ? -mean : 0.0f);
      } else {
        mp = f2(c.has(k, 0) ? -mean : 0.0f, c.has(k, 1) ? -mean : 0.0f);
        mq = f2(c.has(k, 2) ? -mean : 0.0f, c.has(k, 3) ? -mean : 0.0f);
      }
      x[2 * k] = x[2 * k] + mp;
      x[2 * k + 1] = x[2 * k + 1] + mq;
      a = fma2(x[2 * k], x[2 * k], a);
      b = fma2(x[2 * k + 1], x[2 * k + 1], b);
    }
  }
  s[0] = both(a + b);
  team_sum<1>(s, T, team, scratch + 32);       // another part: no barrier between the reads and these writes
  *mean_out = mean;
  *var_out = s[0] * inv_n;
  *rstd_out = rsqrtf(fmaf(s[0], inv_n, eps));  // within 2 units in the last place
}

template <int TX, typename F>
__global__ void __launch_bounds__(kBlock, 1)
    layer_norm_kernel(const __grid_constant__ LayerNormJob j, const __grid_constant__ RowShape r) {
  static_assert(F::VEC, "single elements do not go through the ring");
  char* ring = smem();
  __shared__ float scratch[kScratch];
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const float inv_n = 1.0f / static_cast<float>(n);
  const bool idle = team >= r.teams;           // threads behind the last whole team: touch nothing
  float* weight = reinterpret_cast<float*>(ring + r.params);
  const int width = max(T, F::L) * F::V * kChunk;          // columns of a team's slots
  float* bias = weight + width;
  const uint32_t mine = static_cast<uint32_t>(min(team, r.teams - 1) * r.stages * r.stage_bytes);
  const Columns<F> c(t, n);
  const int64_t step = static_cast<int64_t>(gridDim.x) * r.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const int64_t ahead = step * (r.stages - 1);
  const int64_t x_step = step * j.ld_x * elem_bytes(j.x_type), y_step = step * j.ld_y * elem_bytes(j.y_type);
  const char* next = static_cast<const char*>(row_ptr(j.x, row, j.ld_x, j.x_type));
  char* y = static_cast<char*>(row_ptr(j.y, row, j.ld_y, j.y_type));
  const auto fetch = [&](int slot, int64_t which) {
    if (which < j.tokens && !idle) fetch_row<kBytes<TX>, F>(mine + slot * r.stage_bytes, next, j.x, n, t, T);
    copy_commit();
    next += x_step;
  };
  clear_tails(ring, r.teams * r.stages, r.stage_bytes, n * elem_bytes(j.x_type) / 16 * 16, r.stage_bytes);
  for (int s = 0; s + 1 < r.stages; ++s) fetch(s, row + s * step);
  stage_params<F::VEC>(weight, j.weight, j.param_type, n, width, 1.0f);
  stage_params<F::VEC>(bias, j.bias, j.param_type, n, width, 0.0f);
  __syncthreads();
  if (T > 32 && idle) return;
  int slot = 0;
  // threads of one warp leave together: the block's first team decides
  for (int64_t base = row - team; base < j.tokens; base += step, row += step, y += y_step) {
    const bool live = row < j.tokens && !idle;
    fetch(slot == 0 ? r.stages - 1 : slot - 1, row + ahead);
    copy_wait(r.stages - 1);
    arrive_sync<F::VEC>(T, team);
    F2 x[2 * F::V];
    const uint32_t stage = mine + slot * r.stage_bytes;
    if (live) {
#pragma unroll
      for (int k = 0; k < F::V; ++k) read_chunk<TX, F>(stage, j.x_type, c, k, x[2 * k], x[2 * k + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2 * F::V; ++i) x[i] = f2(0.0f);
    }
    slot = slot + 1 == r.stages ? 0 : slot + 1;
    float mean, var, rstd;
    row_stats<F>(x, c, inv_n, j.eps, T, team, scratch, &mean, &var, &rstd);
    const bool doubt = spread_in_doubt(mean, var, kRowSteps);
    if (T <= 32) __syncwarp();                 // every lane has read the slot that the next copy may take
    if (live) {
      if (t == 0) {
        if (j.mean != nullptr) j.mean[row] = mean;
        if (j.rstd != nullptr) j.rstd[row] = rstd;
      }
      const F2 scale = f2(rstd);
#pragma unroll
      for (int k = 0; k < F::V; ++k) {
        F2 wa, wb, ba, bb;
        param_chunk<F>(r.params, c, k, wa, wb);
        param_chunk<F>(r.params + width * 4, c, k, ba, bb);
        x[2 * k] = fma2(x[2 * k] * scale, wa, ba);
        x[2 * k + 1] = fma2(x[2 * k + 1] * scale, wb, bb);
      }
      write_row<F>(y, j.y_type, c, x);
    }
    if (__any_sync(0xffffffffu, doubt))
      redo_row(j, ring + stage, row, live ? n : 0, weight, bias, t, T, team, scratch + 64, doubt, mean, var);
  }
}

// One row a team: straight from memory, no ring, no parameters in shared memory.
// What counts for a few rows is the depth of dependent loads: one. Single elements
// take this way for any number of rows, and there the parameters come after the
// sums, from L1: 48 registers instead of 64 let four rows of 5003 columns share an
// SM instead of three (1031 x 5003: 13.1 -> 11.2 us). Bound there by instructions,
// 51 an element at 0.67 a cycle with types at run time; with fp32 or not at compile
// time 38 at 0.61, 9.0 us, or 9.1 with the settling of rows in doubt. (V = 1: 40 registers, since 32
// spill around the call: 300 x 1001 3.4 us instead of 3.05.)
template <typename F>
constexpr int kRowRegisters = F::V == 1 ? 40 : F::V == 2 ? (F::VEC ? 56 : 40) : F::V == 4 && !F::VEC ? 48 : 64;
// An element type that is fp32 or not at compile time (T32), or known at run time
// only (kAnyType); 16-bit types select between the conversions.
constexpr int kAnyType = -1;
template <int T32>
__device__ __forceinline__ int known_type(int type) {
  return T32 == kAnyType ? type : T32 == 1 ? static_cast<int>(kF32) : type == kF16 ? static_cast<int>(kF16) : static_cast<int>(kBf16);
}
template <typename F, int X32, int P32, int Y32>
__global__ void __maxnreg__(kRowRegisters<F>)
    layer_norm_row_kernel(const __grid_constant__ LayerNormJob j, const __grid_constant__ RowShape r) {
  __shared__ float scratch[kScratch];
  const int x_type = known_type<X32>(j.x_type), p_type = known_type<P32>(j.param_type), y_type = known_type<Y32>(j.y_type);
  constexpr bool kLate = F::V > 1 && !F::VEC;
  const int T = r.T, team = threadIdx.x / T, t = threadIdx.x - team * T;
  const int n = static_cast<int>(j.n);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * r.teams + team;
  const bool live = team < r.teams && row < j.tokens;
  if (T > 32 && !live) return;
  const Columns<F> c(t, live ? n : 0);
  RawRow<F> rx, rw, rb;
  rx.load(row_ptr(j.x, live ? row : 0, j.ld_x, x_type), x_type, c);
  if (!kLate) {
    rw.load(j.weight, p_type, c);
    rb.load(j.bias, p_type, c);
  }
  F2 x[2 * F::V], p[2 * F::V];
  rx.convert(x_type, x);
  float mean, var, rstd;
  row_stats<F>(x, c, 1.0f / static_cast<float>(n), j.eps, T, team, scratch, &mean, &var, &rstd);
  const bool doubt = live && spread_in_doubt(mean, var, kRowSteps);
  if (kLate && __any_sync(0xffffffffu, doubt)) {
    const Moments m = settle_row(row_ptr(j.x, live ? row : 0, j.ld_x, x_type), x_type, live ? n : 0, static_cast<float>(n),
                                 t, T, team, scratch + 64, doubt, mean, var);
    mean = m.mean;
    if (doubt) rstd = rsqrtf(m.var + j.eps);
#pragma unroll
    for (int i = 0; i < 2 * F::V; ++i) x[i] = x[i] + f2(-m.less);
  }
  if (live && t == 0) {
    if (j.mean != nullptr) j.mean[row] = mean;
    if (j.rstd != nullptr) j.rstd[row] = rstd;
  }
  const F2 scale = f2(rstd);
#pragma unroll
  for (int i = 0; i < 2 * F::V; ++i) x[i] = x[i] * scale;
  if (j.weight != nullptr) {
    if (kLate) rw.load(j.weight, p_type, c);
    rw.convert(p_type, p);
#pragma unroll
    for (int i = 0; i < 2 * F::V; ++i) x[i] = x[i] * p[i];
  }
  if (j.bias != nullptr) {
    if (kLate) rb.load(j.bias, p_type, c);
    rb.convert(p_type, p);
#pragma unroll
    for (int i = 0; i < 2 * F::V; ++i) x[i] = x[i] + p[i];
  }
  if (!kLate && __any_sync(0xffffffffu, doubt)) {          // before x is written over, where y is x
    redo_row(j, row_ptr(j.x, live ? row : 0, j.ld_x, x_type), row, live ? n : 0, nullptr, nullptr, t, T, team,
             scratch + 64, doubt, mean, var);
    if (doubt) return;
  }
  if (live) write_row<F>(static_cast<char*>(row_ptr(j.y, row, j.ld_y, y_type)), y_type, c, x);
}

// Rows too wide for registers: a block per row, three walks over it (the later
// ones served by L1 and L2). Two blocks an SM, which takes at most 32 registers
// (with 36 and one block 600 x 40000 fp32 took 166 us instead of 137).
__global__ void __launch_bounds__(kWideThreads, 2) layer_norm_wide_kernel(const __grid_constant__ LayerNormJob j) {
  __shared__ float scratch[kScratch];
  const float n = static_cast<float>(j.n);
  for (int64_t row = blockIdx.x; row < j.tokens; row += gridDim.x) {
    const void* x = row_ptr(j.x, row, j.ld_x, j.x_type);
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) s[0] += load_elem(x, c, j.x_type);
    team_sum<1>(s, kWideThreads, 0, scratch);
    float mean = s[0] / n, less = 0.0f;
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      const float v = load_elem(x, c, j.x_type) - mean;
      s[0] = fmaf(v, v, s[0]);
    }
    team_sum<1>(s, kWideThreads, 0, scratch + 32);
    float var = s[0] / n, settled = mean;
    if (spread_in_doubt(mean, var, kRowSteps + n / kWideThreads)) {
      const Moments m = settle_row(x, j.x_type, j.n, n, threadIdx.x, kWideThreads, 0, scratch + 64, true, mean, var);
      settled = m.mean;
      var = m.var;
      less = m.less;
    }
    const float rstd = 1.0f / sqrtf(var + j.eps);
    if (threadIdx.x == 0) {
      if (j.mean != nullptr) j.mean[row] = settled;
      if (j.rstd != nullptr) j.rstd[row] = rstd;
    }
    void* y = row_ptr(j.y, row, j.ld_y, j.y_type);
    for (int64_t c = threadIdx.x; c < j.n; c += kWideThreads) {
      float o = ((load_elem(x, c, j.x_type) - mean) - less) * rstd;
      if (j.weight != nullptr) o *= load_elem(j.weight, c, j.param_type);
      if (j.bias != nullptr) o += load_elem(j.bias, c, j.param_type);
      store_elem(y, c, j.y_type, o);
    }
  }
}

template <int TX, typename F>
cudaError_t launch_fwd(const LayerNormJob& j, const RowShape& r, unsigned grid, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(layer_norm_kernel<TX, F>), &done);
  if (e != cudaSuccess) return e;
  layer_norm_kernel<TX, F><<<grid, r.threads(), smem, s>>>(j, r);
  return counted(cudaGetLastError());
}
// The V of row_shape.
template <int TX>
cudaError_t fwd_by_v(const LayerNormJob& j, const RowShape& r, unsigned grid, size_t smem, cudaStream_t s) {
  if (r.L == 16) {
    switch (r.V) {
      case 2: return launch_fwd<TX, Form<2, true, 16>>(j, r, grid, smem, s);
      case 3: return launch_fwd<TX, Form<3, true, 16>>(j, r, grid, smem, s);
      case 4: return launch_fwd<TX, Form<4, true, 16>>(j, r, grid, smem, s);
      case 5: return launch_fwd<TX, Form<5, true, 16>>(j, r, grid, smem, s);
      case 6: return launch_fwd<TX, Form<6, true, 16>>(j, r, grid, smem, s);
      case 8: return launch_fwd<TX, Form<8, true, 16>>(j, r, grid, smem, s);
    }
    return cudaErrorInvalidConfiguration;
  }
  switch (r.V) {
    case 1: return launch_fwd<TX, Form<1, true>>(j, r, grid, smem, s);
    case 2: return launch_fwd<TX, Form<2, true>>(j, r, grid, smem, s);
    case 3: return launch_fwd<TX, Form<3, true>>(j, r, grid, smem, s);
    case 4: return launch_fwd<TX, Form<4, true>>(j, r, grid, smem, s);
    case 5: return launch_fwd<TX, Form<5, true>>(j, r, grid, smem, s);
    case 6: return launch_fwd<TX, Form<6, true>>(j, r, grid, smem, s);
    case 8: return launch_fwd<TX, Form<8, true>>(j, r, grid, smem, s);
    case 10: return launch_fwd<TX, Form<10, true>>(j, r, grid, smem, s);
    case 12: return launch_fwd<TX, Form<12, true>>(j, r, grid, smem, s);
    case 16: return launch_fwd<TX, Form<16, true>>(j, r, grid, smem, s);
  }
  return cudaErrorInvalidConfiguration;
}
template <bool VEC, int X32, int P32, int Y32>
void launch_rows(const LayerNormJob& j, const RowShape& r, unsigned grid, int threads, cudaStream_t s) {
  if (r.V == 1) layer_norm_row_kernel<Form<1, VEC>, X32, P32, Y32><<<grid, threads, 0, s>>>(j, r);
  else if (r.V == 2) layer_norm_row_kernel<Form<2, VEC>, X32, P32, Y32><<<grid, threads, 0, s>>>(j, r);
  else layer_norm_row_kernel<Form<4, VEC>, X32, P32, Y32><<<grid, threads, 0, s>>>(j, r);
}
template <int X32>
void rows_by_type(const LayerNormJob& j, const RowShape& r, bool p32, bool y32, unsigned grid, int threads, cudaStream_t s) {
  if (p32 && y32) launch_rows<false, X32, 1, 1>(j, r, grid, threads, s);
  else if (p32) launch_rows<false, X32, 1, 0>(j, r, grid, threads, s);
  else if (y32) launch_rows<false, X32, 0, 1>(j, r, grid, threads, s);
  else launch_rows<false, X32, 0, 0>(j, r, grid, threads, s);
}
}  // namespace

cudaError_t launch_layer_norm(const LayerNormJob& j, cudaStream_t s) {
  const bool vec = rows_aligned(j.x, j.ld_x, j.n, j.x_type) && rows_aligned(j.y, j.ld_y, j.n, j.y_type) &&
                   reinterpret_cast<uintptr_t>(j.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(j.bias) % 16 == 0;
  RowShape r;
  // Without the ring: few rows, and single elements, for which the ring's copies
  // and barriers cost more than its lead is worth, but for narrow rows in their
  // thousands, where it is 4 % ahead (8192 x 1001): not worth a second form of every
  // ring kernel. us without and with it:
  //   single elements  1031 x 5003 9.0, 18.7; 2000 x 1001 5.6, 7.1; 8192 x 1001
  //                    20.4, 19.5; 8192 x 4097 53, 72
  //   chunks           200 x 320 2.3, 3.1; 200 x 4096 3.9, 5.1; 300 x 4096 5.6, 5.2;
  //                    600 x 1280 4.2, 3.7
  if ((!vec || j.tokens <= 2 * kSms) && single_row_shape(j.tokens, j.n, &r)) {
    const unsigned grid = static_cast<unsigned>((j.tokens + r.teams - 1) / r.teams);
    const int threads = r.threads();
    if (vec) {                                 // up to two rows an SM: types at run time
      launch_rows<true, kAnyType, kAnyType, kAnyType>(j, r, grid, threads, s);
    } else {
      const bool p32 = j.param_type == kF32, y32 = j.y_type == kF32;
      if (j.x_type == kF32) rows_by_type<1>(j, r, p32, y32, grid, threads, s);
      else rows_by_type<0>(j, r, p32, y32, grid, threads, s);
    }
    return counted(cudaGetLastError());
  }
  if (!vec || !row_shape(RowWant{j.tokens, j.n, true, kFwdMaxV, j.x_type, -1, 2}, &r)) {
    layer_norm_wide_kernel<<<grid_of(j.tokens, 1 << 20), kWideThreads, 0, s>>>(j);
    return counted(cudaGetLastError());
  }
  const unsigned grid = grid_of((j.tokens + r.teams - 1) / r.teams, kSms);
  const size_t smem = static_cast<size_t>(r.params) + 2 * static_cast<size_t>(slot_columns(r)) * sizeof(float);
  if (j.x_type == kF32) return fwd_by_v<kF32>(j, r, grid, smem, s);
  if (j.x_type == kBf16) return fwd_by_v<kBf16>(j, r, grid, smem, s);
  return fwd_by_v<kF16>(j, r, grid, smem, s);
}

}  // namespace intlora

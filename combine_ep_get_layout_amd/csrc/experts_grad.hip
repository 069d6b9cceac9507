// Gradients of the experts' products (gfx950).  With z the pre-activations
// and dz their gradient, for every expert e and the rows r of its segment:
//   gated:   dz = [dh * u * act'(g) | dh * act(g)],  z = [g | u] = x [Wg; Wu]^T
//   linear:  dz = dy * act'(z),                      z = x W^T + b
//   dx[r] = sum_o dz[r][o] W_e[o],  dW_e[o] = sum_r dz[r][o] x[r],  db_e = sum_r dz[r]
// dz is rounded to bf16 once, as the matrix cores take it; db sums the
// unrounded values.
#include "experts.hpp"

namespace ep {

// ---- dz ----------------------------------------------------------------------

// Rows of a work item: as many whole rows as make up to 256 vectors of 8 channels, one a
// thread, or one longer row (16 experts x 2,048 rows x 4096 channels 146 us, eight rows an
// item 170; 1 expert x 512 rows 8.6 and 22 us).  A row of little more than 1,024 channels
// leaves nearly half the threads idle.
__host__ __device__ __forceinline__ int dz_rows(int channels) {
  return channels >= 2048 ? 1 : 2048 / channels;
}

// Reads dy and the pre-activations once and writes dz: bound by memory (62,259 rows,
// 2 x 1408 channels: 166 us, 5.3 TB/s).
template <bool GATED>
__global__ __launch_bounds__(256) void expert_dz(GradArgs a) {
  __shared__ TilePlan plan;
  __shared__ int sums[4];
  const int step = dz_rows(a.N);
  plan_tiles<256>(a.seg, step, plan, sums);
  const int vecs = a.N / 8;
  for (int t = blockIdx.x; t < plan.upto[a.seg.E - 1]; t += gridDim.x) {
    const int e = expert_of(plan, a.seg.E, t);
    int64_t start;
    int count;
    segment_of(a.seg, e, start, count);
    const int row0 = (t - plan.first(e)) * step;
    const int rows = min(count - row0, step);
    for (int i = threadIdx.x; i < rows * vecs; i += 256) {
      const int r = i / vecs, ch = (i - r * vecs) * 8;
      const int64_t row = start + row0 + r;
      float d[8], z[8], o[8];
      unpack8(*(const u32x4*)(a.dy + row * a.N + ch), d);
      const int64_t at = row * (GATED ? 2 : 1) * a.N + ch;
      unpack8(*(const u32x4*)(a.pre + at), z);
      if (GATED) {
        float u[8], du[8];
        unpack8(*(const u32x4*)(a.pre + at + a.N), u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float value, slope;
          act_both(a.act, z[c], value, slope);
          o[c] = d[c] * u[c] * slope;
          du[c] = d[c] * value;
        }
        *(u32x4*)(a.dz_out + at + a.N) = pack8(du);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float value, slope;
          act_both(a.act, z[c], value, slope);
          o[c] = d[c] * slope;
        }
      }
      *(u32x4*)(a.dz_out + at) = pack8(o);
    }
  }
}

// ---- db ----------------------------------------------------------------------

constexpr int kBiasWaves = 16, kBiasRows = 4;

// One workgroup per expert and CH channels: eight channels a thread, 8192 / CH
// rows at a time and four such loads in flight, joined over lanes and LDS in a fixed
// order.
template <int CH>
__global__ __launch_bounds__(kBiasWaves* kWave) void expert_dbias(GradArgs a) {
  __shared__ float part[kBiasWaves][CH];
  constexpr int kLanes = CH / 8, kStep = kBiasWaves * kWave / kLanes;
  const int e = blockIdx.y, c0 = blockIdx.x * CH, lane = lane_id();
  const int r0 = threadIdx.x / kLanes, c = (threadIdx.x % kLanes) * 8;
  int64_t start;
  int count;
  segment_of(a.seg, e, start, count);
  float sum[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) sum[q] = 0.0f;
  if (c0 + c < a.N)
    for (int64_t r = r0; r < count; r += kStep * kBiasRows) {
      u32x4 d8[kBiasRows], z8[kBiasRows];
#pragma unroll
      for (int i = 0; i < kBiasRows; ++i) {  // rows past the end repeat the last one
        const int64_t at = (start + min(r + i * kStep, (int64_t)count - 1)) * a.N + c0 + c;
        d8[i] = *(const u32x4*)(a.dy + at);
        z8[i] = a.act == EP_ACT_NONE ? d8[i] : *(const u32x4*)(a.pre + at);
      }
#pragma unroll
      for (int i = 0; i < kBiasRows; ++i) {
        if (r + i * kStep >= count) break;
        float d[8], z[8];
        unpack8(d8[i], d);
        unpack8(z8[i], z);
        if (a.act != EP_ACT_NONE)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float value, slope;
            act_both(a.act, z[q], value, slope);
            d[q] *= slope;
          }
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += d[q];
      }
    }
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int d = kLanes; d < kWave; d <<= 1) sum[q] += __shfl_xor(sum[q], d);
  if (lane < kLanes)
#pragma unroll
    for (int q = 0; q < 8; ++q) part[threadIdx.x / kWave][c + q] = sum[q];
  __syncthreads();
  if (threadIdx.x < CH && c0 + (int)threadIdx.x < a.N) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBiasWaves; ++w) s += part[w][threadIdx.x];
    a.dbias[(int64_t)e * a.N + c0 + threadIdx.x] = s;
  }
}

// ---- dx ----------------------------------------------------------------------

// dx = dz W: the rows run along the contraction (O channels of dz), the
// weights across it, so they are read transposed from LDS rather than stored
// transposed in memory.  62,259 rows over 32 experts, 2 x 1408 -> 4096: 1.31 ms, 1,100
// TFLOP/s, bound as the forward products (matrix cores 70% busy).
struct DxTile {
  int64_t row;
  int rows, n0;
};

template <class S>
struct Dx {
  typedef ColTile<S::BN, S::KR> Chan;
  typedef RowTile<S::BM, S::KB> Row;
  static constexpr int kSlot = Chan::kBytes + Row::kBytes;
  static constexpr int kPasses = Chan::kPasses + Row::kPasses, kLoads = kPasses;
  
  const GradArgs& a;
  const TilePlan& plan;
  lds_char* lds;
  int nk, nfull, mt, nt;
  int64_t z_bytes, w_bytes;
  Chan w_tile;
  Row z_tile;
  const char *w_base, *z_base;
  typename S::acc_t (*acc)[S::TT];

  __device__ __forceinline__ Dx(const GradArgs& a_, const TilePlan& p, lds_char* l)
      : a(a_), plan(p), lds(l) {
    z_bytes = (int64_t)a.O * 2;
    w_bytes = (int64_t)a.C * 2;
    nk = (a.O + S::KR - 1) / S::KR;
    nfull = a.O / S::KR;
    mt = uniform(plan.upto[a.seg.E - 1]);
    nt = (a.C + S::BN - 1) / S::BN;
  }
  __device__ __forceinline__ DxTile setup(int64_t t) {
    int m, n;
    tile_at(t, mt, nt, m, n);
    const int e = expert_of(plan, a.seg.E, m);
    int64_t start;
    int count;
    segment_at(a.seg, e, start, count);
    const int row0 = (m - uniform(plan.first(e))) * S::BM;
    const int rows = min(count - row0, S::BM);
    const int n0 = n * S::BN;
    w_base = (const char*)a.w + (int64_t)e * a.O * w_bytes + n0 * 2;
    z_base = (const char*)a.dz + (start + row0) * z_bytes;
    w_tile.init((uint32_t)w_bytes, a.C - n0);
    z_tile.init([&](int r) -> uint32_t { return (uint32_t)min(r, rows - 1) * (uint32_t)z_bytes; });
    return DxTile{start + row0, rows, n0};
  }
  __device__ __forceinline__ void load_at(int k, lds_char* buf, int p) {
    if (p < Chan::kPasses)
      w_tile.load(p, w_base + (int64_t)k * S::KR * w_bytes, buf);
    else
      z_tile.template load<1 << 20>(p - Chan::kPasses, z_base + (int64_t)k * S::KB, nullptr,
                                    buf + Chan::kBytes);
  }
  __device__ __forceinline__ void tail_at(int k, lds_char* buf) {
    const int left = a.O - k * S::KR;
    w_tile.load_tail(w_base + (int64_t)k * S::KR * w_bytes, left, buf);
    z_tile.template load_tail<1 << 20>(z_base + (int64_t)k * S::KB, nullptr, left * 2,
                                       buf + Chan::kBytes);
  }
  __device__ __forceinline__ void load(int k, int slot, int p) { load_at(k, lds + slot * kSlot, p); }
  __device__ __forceinline__ void tail(int k, int slot) { tail_at(k, lds + slot * kSlot); }

  __device__ __forceinline__ void epilogue(const DxTile& t, lds_char* base) {
    uint16_t* out = a.dx + t.row * a.C + t.n0;
    const TurnLane<S, S::CT> lane;
    const int ch = lane.wc * S::CT * S::MF + lane.channel;
    turn_out<S, S::CT>(base, *(typename S::acc_t(*)[S::CT][S::TT])acc, [](int) { return 0; },
                       [&](int r, const Turned<S>(&turned)[lane.kBatch], const int(&)[lane.kBatch]) {
#pragma unroll
      for (int b = 0; b < lane.kBatch; ++b) {
        const int row = r + b * lane.kRows;
        if (row < t.rows && t.n0 + ch < a.C) {
          float v[8];
          turned[b].get(0, v);
          *(u32x4*)(out + ((uint32_t)row * (uint32_t)a.C + ch)) = pack8(v);
        }
      }
    });
  }
};

template <class S>
__global__ __launch_bounds__(kGemmThreads, 1) void expert_dx(GradArgs a) {
  typedef Dx<S> D;
  __shared__ __align__(16) char lds[S::STAGES][D::kSlot];
  __shared__ TilePlan plan;
  plan_tiles<kGemmThreads>(a.seg, S::BM, plan, (int*)lds);
  lds_char* base = (lds_char*)&lds[0][0];
  D d(a, plan, base);
  const int64_t tiles = (int64_t)d.mt * d.nt;
  if constexpr (S::STAGES == 2) {
    typename S::acc_t acc[S::CT][S::TT];
    d.acc = acc;
    for (int64_t t = block_place(); t < tiles; t += gridDim.x) {
      const DxTile tile = d.setup(t);
      clear<S>(acc);
      products_deep<S>(
          d.w_tile, d.z_tile, base, d.nk, d.nfull,
          [&](int k, lds_char* buf, int p) { d.load_at(k, buf, p); },
          [&](int k, lds_char* buf) { d.tail_at(k, buf); }, acc);
      d.epilogue(tile, base);
    }
  } else {
    RingEngine<S, typename D::Chan, typename D::Row> engine(base);
    d.acc = engine.acc;
    run_ring<S, S::kChains>(d, engine, base, block_place(), tiles, true);
  }
}

// ---- dW ----------------------------------------------------------------------

// dW_e = dz_e^T x_e: both operands run across the contraction, the segment's
// rows (the same sizes: 1.33 ms, 1,080 TFLOP/s).  One workgroup per tile of one expert; an
// expert without rows gets zeros.  A segment's rows are never split, so few tiles with many
// rows leave most of the chip idle (1 expert, 16,384 rows, dx and dW together: 256 x 256
// channels 117 us, 512 x 512 130, 1024 x 1024 166, 2048 x 2048 255).  Each die takes 32 consecutive tiles in turn, so the workgroups that
// run on it together read the same expert's rows and long experts fall on all
// dies alike.
template <class S>
struct Dw {
  typedef ColTile<S::BN, S::KR> Chan;
  typedef ColTile<S::BM, S::KR> Row;
  static constexpr int kSlot = Chan::kBytes + Row::kBytes;
  static constexpr int kPasses = Chan::kPasses + Row::kPasses, kLoads = kPasses;

  const GradArgs& a;
  lds_char* lds;
  int nk, nfull, e, count, c0, o0;
  int64_t x_bytes, z_bytes;
  Chan x_tile;
  Row z_tile;
  const char *x_base, *z_base;
  typename S::acc_t (*acc)[S::TT];

  __device__ __forceinline__ Dw(const GradArgs& a_, lds_char* l) : a(a_), lds(l) {
    x_bytes = (int64_t)a.C * 2;
    z_bytes = (int64_t)a.O * 2;
  }
  __device__ __forceinline__ int setup(int64_t t) {
    const int ct = (a.C + S::BN - 1) / S::BN, ot = (a.O + S::BM - 1) / S::BM;
    e = uniform((int)(t / (ct * ot)));
    int m, n;
    tile_at(t - (int64_t)e * ct * ot, ot, ct, m, n);
    int64_t start;
    segment_at(a.seg, e, start, count);
    c0 = n * S::BN;
    o0 = m * S::BM;
    nk = (int)(((uint32_t)count + S::KR - 1) / S::KR);
    nfull = count / S::KR;
    x_base = (const char*)a.x + start * x_bytes + c0 * 2;
    z_base = (const char*)a.dz + start * z_bytes + o0 * 2;
    x_tile.init((uint32_t)x_bytes, a.C - c0);
    z_tile.init((uint32_t)z_bytes, a.O - o0);
    return 0;
  }
  __device__ __forceinline__ void load_at(int k, lds_char* buf, int p) {
    if (p < Chan::kPasses)
      x_tile.load(p, x_base + (int64_t)k * S::KR * x_bytes, buf);
    else
      z_tile.load(p - Chan::kPasses, z_base + (int64_t)k * S::KR * z_bytes, buf + Chan::kBytes);
  }
  __device__ __forceinline__ void tail_at(int k, lds_char* buf) {
    const int left = count - k * S::KR;
    x_tile.load_tail(x_base + (int64_t)k * S::KR * x_bytes, left, buf);
    z_tile.load_tail(z_base + (int64_t)k * S::KR * z_bytes, left, buf + Chan::kBytes);
  }
  __device__ __forceinline__ void load(int k, int slot, int p) { load_at(k, lds + slot * kSlot, p); }
  __device__ __forceinline__ void tail(int k, int slot) { tail_at(k, lds + slot * kSlot); }

  __device__ __forceinline__ void epilogue(int, lds_char* base) {
    uint16_t* out = a.dw + ((int64_t)e * a.O + o0) * a.C + c0;
    const TurnLane<S, S::CT> lane;
    const int ch = lane.wc * S::CT * S::MF + lane.channel;
    turn_out<S, S::CT>(base, *(typename S::acc_t(*)[S::CT][S::TT])acc, [](int) { return 0; },
                       [&](int r, const Turned<S>(&turned)[lane.kBatch], const int(&)[lane.kBatch]) {
#pragma unroll
      for (int b = 0; b < lane.kBatch; ++b) {
        const int row = r + b * lane.kRows;
        if (o0 + row < a.O && c0 + ch < a.C) {
          float v[8];
          turned[b].get(0, v);
          *(u32x4*)(out + ((uint32_t)row * (uint32_t)a.C + ch)) = pack8(v);
        }
      }
    });
  }
};

template <class S>
__global__ __launch_bounds__(kGemmThreads, 1) void expert_dw(GradArgs a) {
  typedef Dw<S> D;
  __shared__ __align__(16) char lds[S::STAGES][D::kSlot];
  lds_char* base = (lds_char*)&lds[0][0];
  D d(a, base);
  constexpr int kRun = 32;
  const int i = blockIdx.x / kXcds;
  const int64_t t = ((int64_t)(i / kRun) * kXcds + blockIdx.x % kXcds) * kRun + i % kRun;
  const int64_t tiles = (int64_t)a.seg.E * ((a.C + S::BN - 1) / S::BN) * ((a.O + S::BM - 1) / S::BM);
  if (t >= tiles) return;
  if constexpr (S::STAGES == 2) {
    typename S::acc_t acc[S::CT][S::TT];
    d.acc = acc;
    d.setup(t);
    clear<S>(acc);
    products_deep<S>(
        d.x_tile, d.z_tile, base, d.nk, d.nfull,
        [&](int k, lds_char* buf, int p) { d.load_at(k, buf, p); },
        [&](int k, lds_char* buf) { d.tail_at(k, buf); }, acc);
    d.epilogue(0, base);
  } else {
    RingEngine<S, typename D::Chan, typename D::Row> engine(base);
    d.acc = engine.acc;
    run_ring<S, false>(d, engine, base, t, t + 1, false);
  }
}

// ---- launches ------------------------------------------------------------------

typedef Shape<grad::Big> Big;
typedef Shape<grad::Medium> Medium;
typedef Shape<grad::Small> Small;
typedef Shape<grad::Square> Square;
typedef Shape<grad::Pair> Pair;

template <int CH>
static void launch_dbias(const GradArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(expert_dbias<CH>, dim3((a.N + CH - 1) / CH, a.seg.E),
                     dim3(kBiasWaves * kWave), 0, st, a);
}

template <class S>
static void launch_dx(const GradArgs& a, hipStream_t st) {
  const int64_t tiles = ((a.rows + S::BM - 1) / S::BM + a.seg.E) * ((a.C + S::BN - 1) / S::BN);
  hipLaunchKernelGGL(expert_dx<S>, dim3((unsigned)min(tiles, (int64_t)dx_slots<S>())),
                     dim3(kGemmThreads), 0, st, a);
}

template <class S>
static void launch_dw(const GradArgs& a, hipStream_t st) {
  const int64_t tiles =
      (int64_t)a.seg.E * ((a.C + S::BN - 1) / S::BN) * ((a.O + S::BM - 1) / S::BM);
  const int64_t run = 32 * kXcds;
  hipLaunchKernelGGL(expert_dw<S>, dim3((unsigned)((tiles + run - 1) / run * run)),
                     dim3(kGemmThreads), 0, st, a);
}

hipError_t launch_expert_grad(const GradArgs& a, hipStream_t st) {
  if (a.dz_out && a.rows > 0) {
    const int64_t items = a.rows / dz_rows(a.N) + a.seg.E;
    const dim3 grid((unsigned)min(items, (int64_t)kCus * 8));
    if (a.gated)
      hipLaunchKernelGGL(expert_dz<true>, grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL(expert_dz<false>, grid, dim3(256), 0, st, a);
  }
  if (a.dbias) {
    switch (choose_dbias(a.seg.E, a.rows, a.N)) {
      case 32: launch_dbias<32>(a, st); break;
      case 64: launch_dbias<64>(a, st); break;
      default: launch_dbias<256>(a, st);
    }
  }
  if (a.dx && a.rows > 0) {
    switch (choose_dx(a.seg.E, a.rows, a.C, a.O)) {
      case kDxSmall: launch_dx<Small>(a, st); break;
      case kDxMedium: launch_dx<Medium>(a, st); break;
      case kDxBig: launch_dx<Big>(a, st); break;
    }
  }
  if (a.dw) {
    switch (choose_dw(a.seg.E, a.C, a.O)) {
      case kDwBig: launch_dw<Big>(a, st); break;
      case kDwSquare: launch_dw<Square>(a, st); break;
      case kDwPair: launch_dw<Pair>(a, st); break;
    }
  }
  return hipGetLastError();
}

}  // namespace ep

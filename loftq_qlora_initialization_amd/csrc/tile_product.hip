// The tiled product of the adapted layer on the matrix cores: C = X W^T + keep(S V^T)
// for operands whose K runs along their rows, in bf16 or in MXFP4.
//
// A K step is 128 bytes of a row in either format (64 bf16 or 256 FP4 values) and a lane's
// operand of one matrix instruction 16 bytes, so both formats share every address: for
// v_mfma_f32_32x32x16_bf16 lane L supplies row L%32, k = 8 (L/32) .. + 7, for
// v_mfma_scale_f32_32x32x64_f8f6f4 row L%32, k = 32 (L/32) .. + 31, one whole MXFP4 block,
// whose scale byte the instruction applies.  The weight is the first operand, so lane L
// receives token L%32, features 8 (v/4) + 4 (L/32) + v%4 in element v: four consecutive
// features a quad.
//
// A workgroup owns TM tokens x TN features.  Each step's rows go straight from memory to
// LDS (16 bytes a lane).  LDS has 64 banks of 4 bytes, two rows of a
// step: 16-byte piece c of row i lies at place c ^ (i / 2 % 8), so that any 16 rows read
// at one k meet every bank once (c ^ (i % 8) put two of them on each).
//
// Bound by power and by the loads: with random operands the matrix instructions alone reach
// 1.8 (32 x 32) and 2.1 PFLOP/s (16 x 16) in bf16 and 8.0 in FP4 before the clock drops, and
// in the loop the clock stands at 1.75 to 1.85 GHz with the matrix cores busy 51 to 59 % of
// the cycles; what a step waits for is its loads (without them a 256 x 256 step of FP4 takes
// 1.4 instead of 1.9 us).  Traced, mean and least of ten launches: 8192 x 11008 outputs, K =
// 4096: 668 and 665 us, 1.11 PFLOP/s (the library's product of these sizes, in the same trace:
// 688 and 667); 2048 x 4096, K = 11008: 163 and 156 us, 1.13 (172 and 172); 2048 x 11008, K =
// 4096, with the three adapter steps of r = 64: 169 and 159 us, 1.09 (161 and 156, without
// them); FP4 8192 x 28672, K = 8192: 1.08 and 1.05 ms, 3.57 PFLOP/s.  Tried and slower: half steps in a ring of four (64-byte pieces of lines: every
// line is fetched twice), the reads of a quarter step before its products (all waves read,
// then all multiply), 16 x 16 instructions in FP4 (the scales of twice the rows: 77 against 67
// us at 2048 x 11008, K = 4096).
#include "buffer.h"
#include "layer.h"

#include <type_traits>

namespace loftq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 128;

template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (N > 0) {
    static_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// the largest divisor of n that is at most `most` (0: none)
constexpr int divisor_up_to(int n, int most) {
  int d = most < n ? most : n;
  while (d > 1 && n % d != 0) --d;
  return d;
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// Workgroups are dealt to the 8 XCDs round-robin by id; each XCD gets a contiguous run of
// tiles where every tile has one workgroup.  (The K ranges of a divided product are neighbours
// by id, so that its tiles fall to the XCDs otherwise: it has at most two workgroups a CU, and
// its time is its launch, first loads and join.)  Within a run, kBand token tiles by all features in turn, tokens inner, so that
// the rows a band shares stay in the XCD's L2.
constexpr int64_t kBand = 8;
__device__ __forceinline__ void tile_of(int64_t wg, int64_t ntm, int64_t ntn, int64_t& tm, int64_t& tn) {
  const int64_t total = ntm * ntn, per = total / 8;
  const int64_t t = wg < per * 8 ? (wg % 8) * per + wg / 8 : wg;
  const int64_t band = t / (kBand * ntn), first = band * kBand;
  const int64_t height = ntm - first < kBand ? ntm - first : kBand;
  const int64_t in = t - band * kBand * ntn;
  tm = first + in % height;
  tn = in / height;
}

// The rows of a tile in LDS and the loop over K steps that multiplies them with D x D
// matrix instructions (D 16 or 32).  LDS is a ring of R steps.  While one operand set of a
// step is multiplied, the next one is read from LDS; a step's last set is multiplied after
// the barrier that frees its place, while the first operands of the next step are read and
// the loads of step k + R begin to fill that place.
template <int TM, int TN, int WM, int WN, int D, int R>
struct Tile {
  static constexpr int kThreads = (TM / WM) * (TN / WN) * 64;
  static constexpr int MT = WM / D, NT = WN / D;     // D x D tiles of a wave
  static constexpr int kPhases = D / 8, kQuads = D == 32 ? 4 : 1;   // operand sets of a step
  typedef float frag_acc __attribute__((ext_vector_type(kQuads * 4)));
  static constexpr int kRows = TM + TN;              // LDS rows: features, then tokens
  static constexpr int kBuf = kRows * kStepBytes;
  static constexpr int kLoadsW = TN * 8 / kThreads, kLoadsX = TM * 8 / kThreads, kLoads = kLoadsW + kLoadsX;
  // products from one load to the next: close together where a step's loads have one step's
  // time, further apart in a deeper ring (2048 x 4096, K = 11008: 169 -> 163 us)
  static constexpr int kProducts = kPhases * NT * MT;
  static constexpr int kEvery = R > 2 && kProducts >= 4 * kLoads ? 4 : (kProducts >= 2 * kLoads ? 2 : 1);
  static_assert(TN * 8 % kThreads == 0 && TM * 8 % kThreads == 0, "whole 16-byte pieces of either operand per thread");
  static_assert(kProducts >= kLoads * kEvery, "a step's products take its loads between them");
  typedef frag_acc Acc[NT][MT];

  char* lds;
  int tid, lane, w, wm, wn, li, lh;
  int64_t m0, n0, M, N;
  const char *wsrc, *xsrc;      // the next step's first bytes of the tile's rows
  uint32_t off[kLoads];         // this thread's pieces from there
  int left;                     // steps still to load
  int wo, xo;                   // this lane's first operand bytes, features and tokens

  __device__ __forceinline__ Tile(char* lds_, int64_t m0_, int64_t n0_, int64_t M_, int64_t N_)
      : lds(lds_), m0(m0_), n0(n0_), M(M_), N(N_) {
    tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wm = w % (TM / WM), wn = w / (TM / WM);
    li = lane % D, lh = lane / D;
    const int place = (lh ^ (li >> 1 & 7)) << 4;
    wo = (wn * WN + li) * kStepBytes + place;
    xo = (TN + wm * WM + li) * kStepBytes + place;
  }
  // the first step of two operands; rows past the last repeat it (loaded, never stored)
  __device__ __forceinline__ void start(const void* W, int64_t ldw, const void* X, int64_t ldx) {
    wsrc = static_cast<const char*>(W) + n0 * ldw;
    xsrc = static_cast<const char*>(X) + m0 * ldx;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool feature = i < kLoadsW;
      const int c = (feature ? i : i - kLoadsW) * kThreads + tid, row = c >> 3, piece = (c & 7) ^ (row >> 1 & 7);
      const int64_t last = feature ? N - 1 - n0 : M - 1 - m0;
      off[i] = static_cast<uint32_t>((row < last ? row : static_cast<int>(last)) * (feature ? ldw : ldx)) + piece * 16;
    }
  }
  // piece i of the loads of a step into ring place `to`
  __device__ __forceinline__ void load(int to, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        buffer_at(i < kLoadsW ? wsrc : xsrc, left > 0),
        (__attribute__((address_space(3))) void*)(lds + to * kBuf + (i * kThreads + w * 64) * 16), 16, off[i], 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    wsrc += kStepBytes;
    xsrc += kStepBytes;
    --left;
  }
  // operand i of set ph, in the order in which the products ask for them: feature tile 0,
  // the token tiles, the other feature tiles
  template <int ph, int i>
  __device__ __forceinline__ void read(int from, i32x4 (&wf)[NT], i32x4 (&xf)[MT]) {
    const char* t = lds + from * kBuf;
    if constexpr (i == 0)
      wf[0] = *reinterpret_cast<const i32x4*>(t + (wo ^ (ph * (64 / D) << 4)));
    else if constexpr (i <= MT)
      xf[i - 1] = *reinterpret_cast<const i32x4*>(t + (xo ^ (ph * (64 / D) << 4)) + (i - 1) * D * kStepBytes);
    else
      wf[i - MT] = *reinterpret_cast<const i32x4*>(t + (wo ^ (ph * (64 / D) << 4)) + (i - MT) * D * kStepBytes);
  }
  // Every wave has read the place that is loaded next, and all but the last `behind` loads
  // of every wave are done.  Over MXFP4 the scales' loads are among the last ones, so that the
  // ring of three waits for some of the next step's loads as well.
  template <int behind>
  __device__ __forceinline__ void turn() {
    __builtin_amdgcn_sched_barrier(0);
    static_assert(behind < 64, "the counter has six bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(behind) : "memory");
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // `mul(ph, a, b, w, x)` multiplies tile (a, b) of operand set ph; `next()` runs where a step
  // ends.  One copy of the loop's body and no branch in it: the compiler gathers products
  // behind a branch, and more copies cost it registers.
  template <typename Mul, typename Next>
  __device__ __forceinline__ void loop(int steps, Mul&& mul, Next&& next) {
    i32x4 wf[2][NT], xf[2][MT];
    // The products of one operand set, and between them the reads of the next set (from ring
    // place `from`) and loads (into place `to`): issued by themselves, either would keep the
    // matrix cores waiting for all waves of the workgroup at once.
    auto products = [&](auto ph_, int from, int to) __attribute__((always_inline)) {
      constexpr int ph = decltype(ph_)::value, set = ph & 1;
      static_for<NT * MT>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value, at = (ph + 1) % kPhases * NT * MT + i;
        mul(ph_, i / MT, i % MT, wf[set][i / MT], xf[set][i % MT]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (i < NT + MT) read<(ph + 1) % kPhases, i>(from, wf[set ^ 1], xf[set ^ 1]);
        if constexpr (at % kEvery == kEvery - 1 && at / kEvery < kLoads) load(to, at / kEvery);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (NT + MT > NT * MT)
        static_for<NT + MT - NT * MT>([&](auto i_) __attribute__((always_inline)) {
          read<(ph + 1) % kPhases, NT * MT + decltype(i_)::value>(from, wf[set ^ 1], xf[set ^ 1]);
        });
    };
    // loads that a step issues while its last set is multiplied, the first ones of step k + R
    constexpr int kFirst = NT * MT / kEvery < kLoads ? NT * MT / kEvery : kLoads;
    left = steps;
    turn<0>();   // the ring is free
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int i = 0; i < (j < R - 1 ? kLoads : kFirst); ++i) load(j, i);
      if (j < R - 1) advance();
    }
    turn<(R - 2) * kLoads + kFirst>();
    int at = 0, before = R - 1;   // ring places of the step that is multiplied and of the one before
    static_for<NT + MT>([&](auto i_) __attribute__((always_inline)) { read<0, decltype(i_)::value>(0, wf[0], xf[0]); });
    for (int k = 0; k < steps; ++k) {
      // its operand sets but the last, with the rest of the loads of step k - 1 + R
      static_for<kPhases - 1>([&](auto ph_) __attribute__((always_inline)) { products(ph_, at, before); });
      advance();
      turn<(R - 2) * kLoads>();   // step k + 1 has landed
      before = at;
      at = at + 1 == R ? 0 : at + 1;
      products(std::integral_constant<int, kPhases - 1>{}, at, before);
      next();
    }
    turn<0>();
  }
};

template <bool kMx, int TM, int TN, int WM, int WN, int D, int R, typename O>
__global__ __launch_bounds__((TM / WM) * (TN / WN) * 64) void tile_product_kernel(TileProduct t) {
  typedef Tile<TM, TN, WM, WN, D, R> T;
  constexpr int MT = T::MT, NT = T::NT;
  __shared__ __align__(16) char lds[R * T::kBuf];
  const int64_t ntm = (t.M + TM - 1) / TM, ntn = (t.N + TN - 1) / TN;
  int64_t tm, tn;
  const int split = static_cast<int>(blockIdx.x % t.splits);
  tile_of(blockIdx.x / t.splits, ntm, ntn, tm, tn);
  // this workgroup's K steps
  const int per = (t.steps + t.splits - 1) / t.splits, k0 = split * per;
  const int steps = t.steps - k0 < per ? t.steps - k0 : per;
  T g(lds, tm * TM, tn * TN, t.M, t.N);
  const int64_t mw = g.m0 + g.wm * WM + g.li, nw = g.n0 + g.wn * WN;   // this lane's first token, the wave's first feature

  typename T::Acc acc;
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int v = 0; v < 4 * T::kQuads; ++v) acc[a][b][v] = 0.f;
  auto mul_bf16 = [&](auto, int a, int b, i32x4 w, i32x4 x) __attribute__((always_inline)) {
    if constexpr (D == 32)
      acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x),
                                                          acc[a][b], 0, 0, 0);
    else
      acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x),
                                                          acc[a][b], 0, 0, 0);
  };
  auto nothing = []() __attribute__((always_inline)) {};

  // the adapter's term first, in the same accumulators: what the mask drops is cleared
  // before the base's product is added to it
  if (t.adapter_steps > 0 && split == 0) {
    g.start(t.V, t.adapter_steps * kStepBytes, t.S, t.adapter_steps * kStepBytes);
    g.loop(t.adapter_steps, mul_bf16, nothing);
    if (t.drop.thr != 0) {   // N % 4 == 0: a lane's four features share one word
      const uint64_t key = drop_key(t.drop);
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
          for (int q = 0; q < T::kQuads; ++q) {
            const uint64_t word =
                drop_word(key, static_cast<uint64_t>((mw + b * D) * t.N + nw + a * D + 8 * q + 4 * g.lh) >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!drop_keeps(word, j, t.drop.thr)) acc[a][b][4 * q + j] = 0.f;
          }
    }
  }

  g.start(static_cast<const char*>(t.W) + static_cast<int64_t>(k0) * kStepBytes, t.ldw,
          static_cast<const char*>(t.X) + static_cast<int64_t>(k0) * kStepBytes, t.ldx);
  if constexpr (kMx) {
    // each lane's 8 scale bytes of its rows for the step; the operand of matrix
    // instruction kk covers blocks 2 kk + L/32, so byte kk of the bytes that `sel` takes
    const char* wsc = reinterpret_cast<const char*>(t.wscale) + k0 * t.N * 8;
    const char* xsc = reinterpret_cast<const char*>(t.xscale) + k0 * t.M * 8;
    uint32_t wat[NT], xat[MT];
    u32x2 wnext[NT], xnext[MT];
    uint32_t ws[NT], xs[MT];
    const uint32_t sel = g.lh ? 0x07050301u : 0x06040200u;
    int left = steps;
    auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < NT; ++a) wnext[a] = __builtin_amdgcn_raw_buffer_load_b64(buffer_at(wsc, left > 0), wat[a], 0, 0);
#pragma unroll
      for (int b = 0; b < MT; ++b) xnext[b] = __builtin_amdgcn_raw_buffer_load_b64(buffer_at(xsc, left > 0), xat[b], 0, 0);
      wsc += t.N * 8;
      xsc += t.M * 8;
      --left;
    };
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int64_t n = nw + a * D + g.li;
      wat[a] = static_cast<uint32_t>((n < t.N ? n : t.N - 1) * 8);
    }
#pragma unroll
    for (int b = 0; b < MT; ++b) {
      const int64_t m = mw + b * D;
      xat[b] = static_cast<uint32_t>((m < t.M ? m : t.M - 1) * 8);
    }
    fetch();
    auto take = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < NT; ++a) ws[a] = __builtin_amdgcn_perm(wnext[a][1], wnext[a][0], sel);
#pragma unroll
      for (int b = 0; b < MT; ++b) xs[b] = __builtin_amdgcn_perm(xnext[b][1], xnext[b][0], sel);
      fetch();
    };
    take();
    g.loop(
        steps,
        [&](auto ph_, int a, int b, i32x4 w, i32x4 x) __attribute__((always_inline)) {
          constexpr int kk = decltype(ph_)::value;
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              widen(w), widen(x), acc[a][b], 4, 4, kk, static_cast<int>(ws[a]), kk, static_cast<int>(xs[b]));
        },
        take);
  } else {
    g.loop(steps, mul_bf16, nothing);
  }

  // Out through LDS: a lane's four features of a token are 8 or 16 bytes, and stored from
  // there they would touch 32 rows an instruction; each wave turns its outputs round in
  // its share of the tile buffers (16-byte pieces placed as the operands are) and stores
  // whole runs of a token's features.
  constexpr int kRowBytes = WN * static_cast<int>(sizeof(O)), kPieces = kRowBytes / 16;
  constexpr int kShare = R * T::kBuf / (T::kThreads / 64) / 16 * 16;
  constexpr int kB = divisor_up_to(MT, kShare / (D * kRowBytes));   // D-token groups at a time
  static_assert(kB >= 1 && kPieces >= 4 && 64 % kPieces == 0, "a wave's outputs pass through its share");
  auto place = [](int row, int piece) __attribute__((always_inline)) {
    constexpr int kSame = kPieces < 16 ? 16 / kPieces : 1;   // rows that meet all banks together
    return row * kRowBytes + ((piece ^ (row / kSame % (kPieces < 16 ? kPieces : 16))) << 4);
  };
  constexpr int kPer = 16 / static_cast<int>(sizeof(O));
  typedef O piece_t __attribute__((ext_vector_type(kPer)));
  __syncthreads();
  char* share = lds + g.w * kShare;
#pragma unroll
  for (int b0 = 0; b0 < MT; b0 += kB) {
#pragma unroll
    for (int b = b0; b < b0 + kB; ++b)
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int q = 0; q < T::kQuads; ++q) {
          const int row = (b - b0) * D + g.li, f = a * D + 8 * q + 4 * g.lh;
          const f32x4 y = {acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
          if constexpr (sizeof(O) == 4)
            *reinterpret_cast<f32x4*>(share + place(row, f / 4)) = y;
          else
            *reinterpret_cast<bf16x4*>(share + place(row, f / 8) + (f % 8) * 2) =
                bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]), static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
        }
#pragma unroll
    for (int i = 0; i < kB * D * kPieces / 64; ++i) {
      const int row = i * (64 / kPieces) + g.lane / kPieces, piece = g.lane % kPieces;
      const piece_t y = *reinterpret_cast<const piece_t*>(share + place(row, piece));
      const int64_t m = g.m0 + g.wm * WM + b0 * D + row, n = nw + piece * kPer;
      if (m >= t.M) continue;
      O* out = static_cast<O*>(t.out) + (split * t.M + m) * t.N + n;
      if (t.N % kPer == 0) {
        if (n < t.N) *reinterpret_cast<piece_t*>(out) = y;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (n + j < t.N) out[j] = y[j];
      }
    }
  }
}

// out = the sum of `splits` partial products, in the order of their K ranges
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partials, int splits, int64_t n,
                                                   O* __restrict__ out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (n % 4 == 0) {
    f32x4 y = *reinterpret_cast<const f32x4*>(partials + i);
    for (int s = 1; s < splits; ++s) y += *reinterpret_cast<const f32x4*>(partials + s * n + i);
    if constexpr (sizeof(O) == 4)
      *reinterpret_cast<f32x4*>(out + i) = y;
    else
      *reinterpret_cast<bf16x4*>(out + i) = bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]),
                                                   static_cast<__bf16>(y[2]), static_cast<__bf16>(y[3])};
    return;
  }
  for (int64_t j = i; j < i + 4 && j < n; ++j) {
    float y = partials[j];
    for (int s = 1; s < splits; ++s) y += partials[s * n + j];
    out[j] = static_cast<O>(y);
  }
}

// The name under which launch timing files a product: its format and its tile.
template <bool kMx, int TM>
constexpr const char* product_name() {
  if constexpr (kMx) return TM == 256 ? "mx_product_256x256" : TM == 192 ? "mx_product_192x256" : TM == 128 ? "mx_product_128x256" : "mx_product_64x128";
  else return TM == 256 ? "bf16_product_256x256" : TM == 192 ? "bf16_product_192x256" : TM == 128 ? "bf16_product_128x256" : "bf16_product_64x128";
}

template <bool kMx, int TM, int TN, int WM, int WN, int D, int R>
hipError_t launch_tile(const TileProduct& t, hipStream_t s) {
  const int64_t wgs = ((t.M + TM - 1) / TM) * ((t.N + TN - 1) / TN) * t.splits;
  const dim3 grid(static_cast<unsigned>(wgs)), block((TM / WM) * (TN / WN) * 64);
  if (t.odt == LOFTQ_BF16)
    LQ_LAUNCH((product_name<kMx, TM>()), (tile_product_kernel<kMx, TM, TN, WM, WN, D, R, __bf16>), grid, block, 0, s, t);
  else
    LQ_LAUNCH((product_name<kMx, TM>()), (tile_product_kernel<kMx, TM, TN, WM, WN, D, R, float>), grid, block, 0, s, t);
  return hipGetLastError();
}

constexpr int kCUs = 256, kMostSplits = 16;

// Tiles (tokens x features), and what one workgroup's step and the rest of a tile (first
// loads, output) take, in microseconds, measured with every CU at work.  Large tiles read
// less per product, small ones divide a small problem among more CUs.
struct TileShape {
  int tm, tn, per_cu;
  float step_bf16, step_mx, rest;
};
constexpr TileShape kShapes[] = {
    {256, 256, 1, 1.54f, 1.87f, 9.f},
    {192, 256, 1, 1.20f, 1.45f, 9.f},
    {128, 256, 1, 0.80f, 1.06f, 8.f},
    {64, 128, 2, 0.50f, 0.69f, 8.f},
};

}  // namespace

// The shape and the number of K ranges with the least estimated time: rounds of
// workgroups over the CUs, and for more than one range the pass that joins them.
TilePlan plan_tile_product(int64_t M, int64_t N, int steps, int adapter_steps, bool mx) {
  TilePlan best{0, 1};
  float least = 0.f;
  if (steps < 1) return best;
  for (int i = 0; i < 4; ++i) {
    const TileShape& c = kShapes[i];
    const int64_t tiles = ((M + c.tm - 1) / c.tm) * ((N + c.tn - 1) / c.tn);
    const int slots = kCUs * c.per_cu;
    for (int want = 1; want <= kMostSplits; ++want) {
      const int per = (steps + want - 1) / want, splits = (steps + per - 1) / per;
      if (want > 1 && (splits != want || tiles * want > slots)) continue;
      const float rounds = static_cast<float>((tiles * splits + slots - 1) / slots);
      float us = rounds * (c.rest + adapter_steps * c.step_bf16 + per * (mx ? c.step_mx : c.step_bf16));
      if (splits > 1) us += 4.f + static_cast<float>(M * N) * 4.f * (splits + 1) / 4e6f;
      if ((i == 0 && want == 1) || us < least) {
        least = us;
        best = TilePlan{i, splits};
      }
    }
  }
  return best;
}

// Fewer tokens may be divided into more K ranges, so the partials do not grow with M: for each
// shape and number of ranges, the most tokens that it can be chosen for.
size_t tile_product_partial_bound(int64_t M, int64_t N, int steps) {
  size_t most = 0;
  if (steps < 1 || N < 1) return most;
  for (const TileShape& c : kShapes)
    for (int want = 2; want <= kMostSplits; ++want) {
      const int per = (steps + want - 1) / want;
      if ((steps + per - 1) / per != want) continue;
      const int64_t tokens = kCUs * c.per_cu / (want * ((N + c.tn - 1) / c.tn)) * c.tm;
      const size_t bytes = static_cast<size_t>(want * (tokens < M ? tokens : M) * N) * 4;
      if (bytes > most) most = bytes;
    }
  return most;
}

bool tile_product_shape_ok(int64_t M, int64_t N, int64_t K) {
  // one launch has at most 2^32 work-items (256 per 64 x 128 outputs), and 32-bit offsets reach
  // a tile's 256 rows (of 2 K bytes at most) and a step's scales
  return ((M + 63) / 64) * ((N + 127) / 128) < (int64_t(1) << 24) && K < (int64_t(1) << 22) &&
         M < (int64_t(1) << 29) && N < (int64_t(1) << 29);
}

hipError_t launch_tile_product(TileProduct t, bool mx, float* partials, hipStream_t s) {
  const TilePlan p = plan_tile_product(t.M, t.N, t.steps, t.adapter_steps, mx);
  void* const out = t.out;
  const loftq_dtype_t odt = t.odt;
  t.splits = p.splits;
  if (p.splits > 1) {
    t.out = partials;
    t.odt = LOFTQ_F32;
  }
  // 16 x 16 matrix instructions draw less power than 32 x 32 ones (2.11 against 1.79 PFLOP/s of
  // bf16 products alone), but 256 x 256 has no registers for their operands; an MXFP4 lane
  // would need the scales of twice the rows
  hipError_t e;
  switch (p.shape) {
    case 0: e = mx ? launch_tile<true, 256, 256, 64, 128, 32, 2>(t, s) : launch_tile<false, 256, 256, 128, 64, 32, 2>(t, s); break;
    case 1: e = mx ? launch_tile<true, 192, 256, 96, 64, 32, 2>(t, s) : launch_tile<false, 192, 256, 96, 64, 16, 2>(t, s); break;
    case 2: e = mx ? launch_tile<true, 128, 256, 64, 64, 32, 3>(t, s) : launch_tile<false, 128, 256, 64, 64, 16, 3>(t, s); break;
    default: e = mx ? launch_tile<true, 64, 128, 32, 64, 32, 3>(t, s) : launch_tile<false, 64, 128, 32, 64, 16, 3>(t, s); break;
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t n = t.M * t.N;
  const dim3 grid(static_cast<unsigned>((n + 1023) / 1024));
  if (odt == LOFTQ_BF16)
    LQ_LAUNCH("join_product", (join_kernel<__bf16>), grid, dim3(256), 0, s, partials, p.splits, n, static_cast<__bf16*>(out));
  else
    LQ_LAUNCH("join_product", (join_kernel<float>), grid, dim3(256), 0, s, partials, p.splits, n, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace loftq

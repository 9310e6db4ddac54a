// Products of two MXFP4 matrices, out = a b^T, by the scaled matrix
// instructions: every product of two elements is exact, the block scales
// enter inside the instruction, and the sums are float32.
#include "mx_gemm.hpp"

namespace sffn {
namespace {

// ---------------------------------------------------------------- few rows

// M <= 16 rows of a: one workgroup for 16 rows of b, whose waves share out K
// by 128-wide groups and add their sums in LDS. Each wave has a ring of its
// own in LDS, filled by direct copies kFewSlots groups ahead: loads straight
// into the instruction's lanes, which hold different rows, take an access
// each (16 x 1024 x 16384: 10.5 us, so 5.4). The
// rows of b are the instruction's first operand: lane l holds row l % 16, k =
// 32 (l / 16) .. + 31, and of the result four consecutive n of row m = l % 16.
// A slot holds the 16 rows of b and those of a, row r's 16-byte piece c at
// position c ^ (r / 4) % 4 (so that 16 lanes reading one piece of 16 rows meet
// 16 different bank groups), then their scale dwords.
//
// W waves: 8 for long K, 4 else (1 x 1024 x 16384 5.4 us, with 4 6.3; 1 x 5632
// x 2048 3.35, 2.95; even at K = 4096).
constexpr int kFewSlots = 2;                   // with three 3.1 us for the last
constexpr int kFewSlot = 2 * 1024 + 2 * 256;   // 64 dwords of scales of either
constexpr int kFewRing = kFewSlots * kFewSlot;

template <int W, typename O>
__global__ __launch_bounds__(W * 64) void mx_few_kernel(MxGemmArgs g) {
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kq = lane >> 4, l15 = lane & 15;
  const int64_t rb = mx_padded(g.K) / 2;
  const int G = (int)(rb / 64);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  char* ring = smem + wave * kFewRing;

  // rows past the end repeat the last one
  const int lr = lane >> 2, lc = (lane & 3) ^ ((lane >> 4) & 3);
  const int ma = (int)g.M - 1, nb = (int)min(g.N - 1 - n0, (int64_t)15);
  const uint32_t va = (uint32_t)min(lr, ma) * (uint32_t)rb + lc * 16;
  const uint32_t vb = (uint32_t)min(lr, nb) * (uint32_t)rb + lc * 16;
  const uint32_t vsa = (uint32_t)min(l15, ma) * 4, vsb = (uint32_t)min(l15, nb) * 4;
  const uint8_t* pb = g.b + n0 * rb;
  auto copy = [&](int t, int slot) {
    char* s = ring + slot * kFewSlot;
    copy16(pb + (int64_t)t * 64, vb, s);
    copy16(g.a + (int64_t)t * 64, va, s + 1024);
    copy4(g.b_sc + ((int64_t)t * g.N + n0) * 4, vsb, s + 2048);
    copy4(g.a_sc + (int64_t)t * g.M * 4, vsa, s + 2304);
  };
  f32x4_t acc = {};
  // a wave's groups are wave, wave + W, ..; past the last it copies that
  // again, so that the number of copies in flight is always the same
  const int mine = G > wave ? (G - wave + W - 1) / W : 0;
  const int last = wave + W * (mine - 1);
  if (mine > 0) {
#pragma unroll
    for (int p = 0; p < kFewSlots; ++p) copy(min(wave + W * p, last), p);
    int slot = 0;
    for (int q = 0; q < mine; ++q) {
      // the oldest slot's copies have landed
      wait_point<wait_imm((kFewSlots - 1) * 4, 15)>();
      const char* s = ring + slot * kFewSlot;
      const int c = l15 * 64 + ((kq ^ ((l15 >> 2) & 3)) << 4);
      const i32x4_t bv = *(const i32x4_t*)(s + c), av = *(const i32x4_t*)(s + 1024 + c);
      const int bs = *(const uint8_t*)(s + 2048 + l15 * 4 + kq);
      const int as = *(const uint8_t*)(s + 2304 + l15 * 4 + kq);
      // everything read before the slot is written again
      wait_point<wait_imm(63, 0)>();
      copy(min(wave + W * (q + kFewSlots), last), slot);
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(bv), frag(av), acc, kFp4, kFp4,
                                                             0, bs, 0, as);
      slot = slot + 1 == kFewSlots ? 0 : slot + 1;
    }
  }
  // a wave's ring takes its sums once its copies have landed
  wait_point<wait_imm(0, 0)>();
  *(f32x4_t*)(ring + lane * 16) = acc;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // output (m, n) is value n % 4 of lane 16 (n / 4) + m
  const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
  const char* r = smem + (16 * (n >> 2) + m) * 16 + (n & 3) * 4;
  float sum = *(const float*)r;
#pragma unroll
  for (int w = 1; w < W; ++w) sum += *(const float*)(r + w * kFewRing);
  if (m < g.M && n <= nb) put((O*)g.out + m * g.ldo + n0 + n, sum);
}

// ---------------------------------------------------------------- small tiles

// A (32 I) x 64 tile a workgroup, whose four waves share out K by 128-wide
// groups. With few tiles the time is the latency of the operands' loads, so
// each wave has a ring of its own in LDS, filled by direct copies kMidSlots
// groups ahead (two, which leave room for a second workgroup on the CU: 1024
// x 2048 x 2048 10.2 us, with four 12.1): nothing is shared before the sums, so there is no barrier
// in the loop, only the wave's wait for its own oldest copies. A slot holds
// the rows' codes, row r's 16-byte piece c at position c ^ (r / 4) % 4 (so
// that 16 lanes reading one piece of 16 rows meet 16 different bank
// groups), then their scale dwords. Lane l holds row l % 32 of a 32-row
// block and k = 32 (l / 32) .. + 31 of a 64-wide step.
constexpr int kMidSlots = 2;

template <int I>
struct Mid {
  static constexpr int TM = 32 * I, ROWS = TM + 64;
  static constexpr int SLOT = ROWS * 64 + 512;   // 64 dwords of scales of either operand
  static constexpr int LPS = ROWS / 16 + 2;    // copies a group
  static constexpr int RING = 4 * kMidSlots * SLOT;
  static constexpr int LDS = RING > 4 * TM * 64 * 4 ? RING : 4 * TM * 64 * 4;
};

template <int I, typename O>
__global__ __launch_bounds__(256) void mx_mid_kernel(MxGemmArgs g) {
  typedef Mid<I> C_;
  constexpr int TM = C_::TM, ROWS = C_::ROWS, SLOT = C_::SLOT, LPS = C_::LPS;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hi = lane >> 5, l31 = lane & 31;
  const int64_t rb = mx_padded(g.K) / 2;
  const int G = (int)(rb / 64);
  const int64_t n0 = (int64_t)blockIdx.x * 64, m0 = (int64_t)blockIdx.y * TM;
  char* ring = smem + wave * (kMidSlots * SLOT);

  // rows past the end repeat the last one
  const int lr = lane >> 2, lc = (lane & 3) ^ ((lane >> 4) & 3);
  const int ma = (int)min(g.M - 1 - m0, (int64_t)TM), nb = (int)min(g.N - 1 - n0, (int64_t)64);
  uint32_t va[2 * I], vb[4];
#pragma unroll
  for (int i = 0; i < 2 * I; ++i) va[i] = (uint32_t)min(i * 16 + lr, ma) * (uint32_t)rb + lc * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) vb[i] = (uint32_t)min(i * 16 + lr, nb) * (uint32_t)rb + lc * 16;
  const uint32_t vsa = (uint32_t)min(lane & (TM - 1), ma) * 4;
  const uint32_t vsb = (uint32_t)min(lane, nb) * 4;
  const uint8_t* pa = g.a + m0 * rb;
  const uint8_t* pb = g.b + n0 * rb;
  // (the scales of TM < 64 rows with repetitions)
  auto copy = [&](int t, int slot) {
    char* s = ring + slot * SLOT;
    const int64_t k = (int64_t)t * 64;
#pragma unroll
    for (int i = 0; i < 2 * I; ++i) copy16(pa + k, va[i], s + i * 1024);
#pragma unroll
    for (int i = 0; i < 4; ++i) copy16(pb + k, vb[i], s + TM * 64 + i * 1024);
    copy4(g.a_sc + ((int64_t)t * g.M + m0) * 4, vsa, s + ROWS * 64);
    copy4(g.b_sc + ((int64_t)t * g.N + n0) * 4, vsb, s + ROWS * 64 + 256);
  };
  f32x16_t acc[I][2] = {};
  // a wave's groups are wave, wave + 4, ..; past the last it copies that
  // again, so that the number of copies in flight is always the same
  const int mine = G > wave ? (G - wave + 3) / 4 : 0;
  const int last = wave + 4 * (mine - 1);
  if (mine > 0) {
#pragma unroll
    for (int p = 0; p < kMidSlots; ++p) copy(min(wave + 4 * p, last), p);
    int slot = 0;
    for (int q = 0; q < mine; ++q) {
      // the oldest slot's copies have landed
      wait_point<wait_imm((kMidSlots - 1) * LPS, 15)>();
      const char* s = ring + slot * SLOT;
      i32x4_t av[I][2], bv[2][2];
      uint32_t as[I], bs[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = ((2 * h + hi) ^ ((l31 >> 2) & 3)) * 16;
#pragma unroll
        for (int i = 0; i < I; ++i) av[i][h] = *(const i32x4_t*)(s + (i * 32 + l31) * 64 + c);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          bv[j][h] = *(const i32x4_t*)(s + (TM + j * 32 + l31) * 64 + c);
      }
      // the block of substep h is 2 h + hi: shifted so that byte 2 h is it
#pragma unroll
      for (int i = 0; i < I; ++i)
        as[i] = *(const uint32_t*)(s + ROWS * 64 + (i * 32 + l31) * 4) >> (8 * hi);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        bs[j] = *(const uint32_t*)(s + ROWS * 64 + 256 + (j * 32 + l31) * 4) >> (8 * hi);
      // everything read before the slot is written again
      wait_point<wait_imm(63, 0)>();
      copy(min(wave + 4 * (q + kMidSlots), last), slot);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              frag(av[i][0]), frag(bv[j][0]), acc[i][j], kFp4, kFp4, 0, (int)as[i], 0, (int)bs[j]);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              frag(av[i][1]), frag(bv[j][1]), acc[i][j], kFp4, kFp4, 2, (int)as[i], 2, (int)bs[j]);
        }
      slot = slot + 1 == kMidSlots ? 0 : slot + 1;
    }
  }
  // the rings give way to the waves' sums once every copy has landed
  wait_point<wait_imm(0, 0)>();
  __syncthreads();
  float(*red)[TM * 64] = (float(*)[TM * 64])smem;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        red[wave][(i * 32 + 8 * (e / 4) + 4 * hi + e % 4) * 64 + j * 32 + l31] = acc[i][j][e];
  __syncthreads();
  for (int e = threadIdx.x; e < TM * 64; e += 256) {
    const int64_t m = m0 + e / 64, n = n0 + e % 64;
    if (m < g.M && n < g.N)
      put((O*)g.out + m * g.ldo + n, red[0][e] + red[1][e] + red[2][e] + red[3][e]);
  }
}

// ---------------------------------------------------------------- large tiles

// A (64 MI) x 256 tile a workgroup of 4 waves (2 x 2), a wave (32 MI) x 128
// of it: MI x 4 blocks of the 32 x 32 x 64 instruction. Both operands stream
// through a ring of LDS slots filled by direct copies, 128 k (64 bytes of a
// row, and its four scale bytes) a slot. The ring runs on across the tiles
// of a workgroup. A slot holds the rows' codes, row r's 16-byte piece c at
// position c ^ (r / 4) % 4 (so that 16 lanes reading one piece of 16 rows
// meet 16 different bank groups), then the rows' scale dwords, those of the
// 32-row blocks of a wave's rows side by side: one read gives a lane its
// scales of an operand.
//
// A stage is two substeps of 64 k. Substep 0 multiplies fragments that are
// in registers while those of substep 1 are read; then the wave waits for
// its copies of the next stage, the barrier makes everyone's visible (and
// frees the slot, whose last fragments are in registers), and substep 1
// multiplies while the next stage's first fragments are read. Every
// substep starts half a stage of copies, NSLOT stages ahead.
template <int MI, int NS>
struct Big {
  static constexpr int BM = 64 * MI, BN = 256, WM = 32 * MI;
  static constexpr int NSLOT = NS;
  static constexpr int ROWS = BM + BN;
  static constexpr int SLOT = ROWS * 64 + ROWS * 4;
  static constexpr int LPS = MI + 4 + 2;          // copies a wave and stage
  static constexpr int LDS = NSLOT * SLOT;
  static constexpr int WGS = LDS > 80 * 1024 ? 1 : 2;   // workgroups a CU
};

template <int MI, int NS, typename O>
__global__ __launch_bounds__(256, (Big<MI, NS>::WGS)) void mx_big_kernel(MxGemmArgs g) {
  typedef Big<MI, NS> C_;
  constexpr int BM = C_::BM, BN = C_::BN, NSLOT = C_::NSLOT, SLOT = C_::SLOT, LPS = C_::LPS;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  const int hi = lane >> 5, l31 = lane & 31;
  const int M = (int)g.M, N = (int)g.N;
  const int64_t rb = mx_padded(g.K) / 2;
  const int G = (int)(rb / 64);

  // Tiles in groups of kGroupM row tiles, all column tiles of a group before
  // the next; each XCD takes a contiguous eighth of that order, so that its
  // CUs share row panels in its L2.
  const int mt = (M + BM - 1) / BM, ntl = (N + BN - 1) / BN;
  const int ntiles = mt * ntl;
  const int per = (ntiles + kNXcd - 1) / kNXcd;
  const int t_begin = (blockIdx.x % kNXcd) * per;
  const int t_end = min(ntiles, t_begin + per);
  const int step = gridDim.x / kNXcd;
  int L = t_begin + (int)(blockIdx.x / kNXcd);
  if (L >= t_end) return;
  auto coords = [&](int t, int& m0, int& n0) {
    const int grp = t / (kGroupM * ntl);
    const int gsz = min(mt - grp * kGroupM, kGroupM);
    const int rr = t - grp * kGroupM * ntl;
    m0 = (grp * kGroupM + rr % gsz) * BM;
    n0 = (rr / gsz) * BN;
  };

  // copy state: the tile and stage whose copies go out next. A wave copies
  // rows 16 MI wave .. of A and 64 wave .. of B, 16 rows a copy (lane l row
  // l / 4, piece l % 4 of the slot), and 64 rows' scales of each (of A, with
  // MI = 2, two waves the same ones). Rows past the end repeat the last one.
  const int lr = lane >> 2, lc = (lane & 3) ^ ((lane >> 4) & 3);
  const int asw = MI == 4 ? wave : (wave & 1);
  uint32_t va[MI], vb[4], vsa, vsb;
  const uint8_t *pa, *pb;
  int cm0, cn0, ct = L, ck = 0;
  auto set_tile = [&]() {
    coords(ct, cm0, cn0);
    pa = g.a + (int64_t)cm0 * rb;
    pb = g.b + (int64_t)cn0 * rb;
    const int ma = M - 1 - cm0, nb = N - 1 - cn0;
#pragma unroll
    for (int i = 0; i < MI; ++i)
      va[i] = (uint32_t)min(wave * (16 * MI) + i * 16 + lr, ma) * (uint32_t)rb + lc * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vb[i] = (uint32_t)min(wave * 64 + i * 16 + lr, nb) * (uint32_t)rb + lc * 16;
    const int qa = asw * 64 + lane, qb = wave * 64 + lane;
    vsa = (uint32_t)min(qa / (32 * MI) * C_::WM + qa % MI * 32 + qa / MI % 32, ma) * 4;
    vsb = (uint32_t)min(qb / 128 * 128 + qb % 4 * 32 + qb / 4 % 32, nb) * 4;
  };
  // copy i of the copy state's stage into a slot: MI + 1 of A, 5 of B, the
  // scales last
  auto copy_a = [&](int slot, int i) {
    char* s = smem + slot * SLOT;
    if (i < MI)
      copy16(pa + (int64_t)ck * 64, va[i], s + (wave * (16 * MI) + i * 16) * 64);
    else
      copy4(g.a_sc + ((int64_t)ck * M + cm0) * 4, vsa, s + C_::ROWS * 64 + asw * 256);
  };
  auto copy_b = [&](int slot, int i) {
    char* s = smem + slot * SLOT;
    if (i < 4)
      copy16(pb + (int64_t)ck * 64, vb[i], s + (BM + wave * 64 + i * 16) * 64);
    else
      copy4(g.b_sc + ((int64_t)ck * N + cn0) * 4, vsb,
            s + C_::ROWS * 64 + BM * 4 + wave * 256);
  };
  auto advance = [&]() {
    if (++ck == G) {
      if (ct + step < t_end) {
        ct += step;
        ck = 0;
        set_tile();
      } else {
        ck = G - 1;   // past the last stage: it again, into slots not read
      }
    }
  };

  i32x4_t af[2][MI], bf[2][4];
  uint32_t as[MI], bs[4];
  typedef uint32_t asv_t __attribute__((ext_vector_type(MI)));
  asv_t asn;
  u32x4_t bsn;
  // read i of a substep: MI fragments of A, 4 of B, then the stage's scales
  auto read_one = [&](int slot, int s, int buf, int i) {
    const char* p = smem + slot * SLOT;
    const int c = ((2 * s + hi) ^ ((l31 >> 2) & 3)) * 16;
    if (i < MI)
      af[buf][i] = *(const i32x4_t*)(p + (wr * C_::WM + i * 32 + l31) * 64 + c);
    else if (i < MI + 4)
      bf[buf][i - MI] = *(const i32x4_t*)(p + (BM + wc * 128 + (i - MI) * 32 + l31) * 64 + c);
    else if (i == MI + 4)
      asn = *(const asv_t*)(p + C_::ROWS * 64 + (wr * 32 + l31) * (4 * MI));
    else
      bsn = *(const u32x4_t*)(p + C_::ROWS * 64 + BM * 4 + (wc * 32 + l31) * 16);
  };
  // the block of substep s is 2 s + hi: shifted so that byte 2 s is it
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) as[i] = asn[i] >> (8 * hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) bs[j] = bsn[j] >> (8 * hi);
  };
  f32x16_t acc[MI][4];

  // A substep's 4 MI MFMAs with its R reads and C copies spread over them,
  // one read before each of the first ones and the copies evenly: a burst
  // of either would hold the wave's issue slot while the matrix core idles.
  // (In program order as well: the compiler cannot tell that a copy writes
  // another slot than the reads around it read.)
  auto substep = [&](auto sub, auto reads, auto copies, auto&& read, auto&& copy) {
    constexpr int S = decltype(sub)::value, R = decltype(reads)::value,
                  C = decltype(copies)::value, N = 4 * MI;
    unroll<N>([&](auto kk) {
      constexpr int k = decltype(kk)::value, i = k / 4, j = k % 4;
      constexpr int r0 = k * R / N < R ? (k < N / 2 ? k * R / (N / 2) : R) : R;
      constexpr int r1 = k + 1 <= N / 2 ? (k + 1) * R / (N / 2) : R;
      constexpr int c0 = k * C / N, c1 = (k + 1) * C / N;
      unroll<r1 - r0>([&](auto q) { read(r0 + decltype(q)::value); });
      unroll<c1 - c0>([&](auto q) { copy(c0 + decltype(q)::value); });
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          frag(af[S][i]), frag(bf[S][j]), acc[i][j], kFp4, kFp4, 2 * S, (int)as[i], 2 * S,
          (int)bs[j]);
      if constexpr (r1 > r0) __builtin_amdgcn_sched_group_barrier(0x100, r1 - r0, 0);
      if constexpr (c1 > c0) __builtin_amdgcn_sched_group_barrier(0x010, c1 - c0, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    });
    __builtin_amdgcn_sched_barrier(0);
  };

  set_tile();
#pragma unroll
  for (int p = 0; p < NSLOT - 1; ++p) {
#pragma unroll
    for (int i = 0; i <= MI; ++i) copy_a(p, i);
#pragma unroll
    for (int i = 0; i < 5; ++i) copy_b(p, i);
    advance();
  }
#pragma unroll
  for (int i = 0; i <= MI; ++i) copy_a(NSLOT - 1, i);
  int slot = 0, pslot = NSLOT - 1;
  wait_point<wait_imm((NSLOT - 2) * LPS + MI + 1, 15)>();
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < MI + 6; ++i) read_one(0, 0, 0, i);

  for (;;) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int k = 0; k < G; ++k) {
      const int next = slot + 1 == NSLOT ? 0 : slot + 1;
      wait_point<wait_imm(63, 0)>();   // fragments of substep 0, scales
      take_scales();
      substep(Int<0>{}, Int<MI + 4>{}, Int<5>{}, [&](int i) { read_one(slot, 1, 1, i); },
              [&](int i) { copy_b(pslot, i); });
      advance();
      wait_point<wait_imm((NSLOT - 2) * LPS, 0)>();
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      substep(Int<1>{}, Int<MI + 6>{}, Int<MI + 1>{}, [&](int i) { read_one(next, 0, 0, i); },
              [&](int i) { copy_a(slot, i); });
      pslot = slot;
      slot = next;
    }
    settle_sums<MI>();
    int m0, n0;
    coords(L, m0, n0);
    O* out = (O*)g.out + (int64_t)(m0 + wr * C_::WM + 4 * hi) * g.ldo + n0 + wc * 128 + l31;
    const int mleft = M - (m0 + wr * C_::WM + 4 * hi), nleft = N - (n0 + wc * 128 + l31);
    if (m0 + BM <= M && n0 + BN <= N) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          O* o = out + (int64_t)(i * 32 + 8 * (e / 4) + e % 4) * g.ldo;
#pragma unroll
          for (int j = 0; j < 4; ++j) put(o + j * 32, sum_of<MI>(acc[i][j][e]));
          __builtin_amdgcn_sched_barrier(0);   // not all accumulators into registers first
        }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = i * 32 + 8 * (e / 4) + e % 4;
          O* o = out + (int64_t)r * g.ldo;
          if (r < mleft) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j * 32 < nleft) put(o + j * 32, sum_of<MI>(acc[i][j][e]));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    L += step;
    if (L >= t_end) break;
  }
  // no copy may land after the workgroup's LDS is another's
  wait_point<wait_imm(0, 0)>();
}

// The kernel by the number of tiles, measured with float32 results (us,
// M x N x K; the sides of each border):
//   few rows:    up to 16 (from graphs, on matrices b that the caches do not
//                hold): 1 x 5632 x 2048 3.8, 32 x 64 tiles 4.4; 16 x 20480 x
//                4096 (320 tiles: a second round of the CUs for 64 of them)
//                12.9, 14.3; 2 x 16320 x 16384 30.0, 33.0
//   32 x 64:     for 8 to 16 rows and K from 2048 on where the tiles fill
//                their rounds of the CUs to 7/8, since their copies of a serve
//                64 rows of b, the few rows' 16: 16 x 16384 x 4096 9.2, few
//                rows 10.7; 16 x 65536 x 8192 62.3, 80.6; 8 x 14336 x 2048
//                6.05, 6.37. (4 x 16384 x 16384 33.1, 32.7; 16 x 16320 x 1024
//                4.67, 4.59.) And
//                up to 128 tiles of 64 x 64, which leave CUs without one:
//                256 x 2048 x 2048 (128 tiles) 5.5, 64 x 64 5.8;
//                256 x 4096 x 2048 (256) 6.5, 64 x 64 6.2
//   64 x 64:     up to 512 such tiles, two a CU: 1024 x 2048 x 2048 (512)
//                10.2, 128 x 256 12.3; 512 x 5632 x 2048 (704) 13.4, 13.2
//   128 x 256:   two workgroups a CU, better while a 256 x 256 tile each
//                leaves CUs idle (4096 x 2048 x 5632, 128 of them: 33.0, 256 x
//                256 37.7; 2048 x 5632 x 2048, 176: 23.4, 22.2) and for short K,
//                where one stores while the other multiplies (4096 x 8192 x
//                384: 28.0, 33.1; 4096 x 4096 x 1024: 21.7, 21.5)
//   256 x 256:   8192 x 5632 x 2048 70.5 (2.68 PFLOP/s), 128 x 256 74.8;
//                8192 x 8192 x 8192 268 (4.1), 313. Matrix instructions alone,
//                on random operands, run at 6.0 PFLOP/s here (power).
template <typename O>
hipError_t launch(const MxGemmArgs& g, hipStream_t s) {
  const int64_t m32 = (g.M + 31) / 32, n64 = (g.N + 63) / 64, t64 = (g.M + 63) / 64 * n64;
  const bool filled = 8 * n64 >= 7 * kCus * ((n64 + kCus - 1) / kCus);
  const bool wide = g.M >= 8 && g.M <= 16 && g.K >= 2048 && filled;
  if (g.M <= 16 && !wide) {
    const unsigned grid = (unsigned)((g.N + 15) / 16);
    if (g.K <= 4096) mx_few_kernel<4, O><<<grid, 256, 4 * kFewRing, s>>>(g);
    else mx_few_kernel<8, O><<<grid, 512, 8 * kFewRing, s>>>(g);
    return hipGetLastError();
  }
  const int64_t t256 = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  if (wide || t64 <= 128)
    mx_mid_kernel<1, O><<<dim3((unsigned)n64, (unsigned)m32), 256, Mid<1>::LDS, s>>>(g);
  else if (t64 <= 512 || g.K == 0)   // (no tile of the others is ever empty)
    mx_mid_kernel<2, O><<<dim3((unsigned)n64, (unsigned)((g.M + 63) / 64)), 256, Mid<2>::LDS,
                          s>>>(g);
  else if (t256 <= 160 || g.K <= 1024)
    mx_big_kernel<2, 3, O><<<2 * kCus, 256, Big<2, 3>::LDS, s>>>(g);
  else
    mx_big_kernel<4, 4, O><<<kCus, 256, Big<4, 4>::LDS, s>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(Dtype out_dt, const MxGemmArgs& g, hipStream_t s) {
  return out_dt == kBF16 ? launch<uint16_t>(g, s) : launch<float>(g, s);
}

}  // namespace sffn

// The body of the GEMM kernel (gemm_kernel.h): workgroup `bid` of `nblocks` of the product
// args_in, with template parameters LB, EPI, BM, BN and F8 and LDS_BYTES of LDS in `smem`.

  static_assert((BM == 256 && (BN == 256 || BN == 128)) || (BM == 128 && BN == 128), "tile shapes");
  static_assert(F8 == 0 || LB == KC, "FP8 operands are K-contiguous");
  // Paired products (EPI_F32_PAIR, EPI_F32_ACC_PAIR): two accumulator sets, which
  // only the 256 x 128 and 128 x 128 tiles have registers for.
  constexpr bool PAIR = EPI == EPI_F32_PAIR || EPI == EPI_F32_ACC_PAIR;
  static_assert(!PAIR || (F8 == 0 && BN == 128), "paired products: bf16, 256 x 128 or 128 x 128 tiles");
  static_assert(8 * 64 * ROW_B <= 160 * 1024, "two staging regions per wave fit the LDS");
  constexpr int BK = TILE_BK;
  constexpr int SLOT = 128 * BK * 2;
  constexpr int NA = BM / 128;              // A quarters (128 rows x BK) per K step
  constexpr int NQ = NA + BN / 128;         // quarters loaded per K step
  constexpr int NSLOT = 10;
  constexpr int SPS = BM == 128 ? 2 : 4;    // ring slots per K step
  constexpr int P = 5;                      // ring period in K steps (SPS P = 0 mod 10)
  // Prefetch distance in K steps: as far as the ring allows.  Step k+D takes
  // step k-1's last slots (free once every wave has passed step k-1's mid-step
  // barrier) and, for 256-row tiles, step k's first ones (free after step k's).
  // (Packing 256 x 128 steps into three slots for a distance of 3 needs a
  // period of 10 steps, and measured slower.)
  constexpr int D = BM == 128 ? 4 : 2;
  constexpr int QS0 = BM == 128 ? 1 : 2;    // quarters of step k+D loaded in sub-step 0
  constexpr int FI = BM / 32, FJ = BN / 32;  // 16 x 16 blocks per wave: FI x FJ
  static_assert(BK == 64 && NSLOT * SLOT == LDS_BYTES, "ten 16 KiB slots fill the LDS");

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  int tm, tn, split;
  tile_of(bid, nblocks, args_in.tiles_m, args_in.tiles_n, tm, tn, split);
  // A batched launch is unsplit: the "split" index names the workgroup's product.
  GemmArgs args = args_in;
  if (args_in.batch > 1) {
    const int j = split;
    split = 0;
    args.a = args_in.a_arr[j];
    args.b = args_in.b_arr[j];
    args.out = args_in.out_arr[j];
    args.out2 = args_in.out2_arr[j];
    args.aux = args_in.aux_arr[j];
  }
  if (PAIR) {  // product 0's operands; product 1's are a_arr[1] and b_arr[1]
    args.a = args_in.a_arr[0];
    args.b = args_in.b_arr[0];
  }
  constexpr bool GLU = is_glu(EPI);
  static_assert(!(GLU || is_dglu(EPI)) || F8 == 0, "gated products: bf16");
  const int m0 = tm * BM, n0 = tn * (GLU ? BN / 2 : BN);  // first row and column (EPI_GLU: pair)
  const int k_begin = split * args.k_split;
  const int k_end = min(args.K, k_begin + args.k_split);
  const int nk = (k_end - k_begin + BK - 1) / BK;
  // K steps of the whole loop: product 1 (paired launches) follows product 0's nk.
  const int nk_all = PAIR ? 2 * nk : nk;

  QuarterKC qa[NA], qb[BN / 128];
  QuarterMC qm[BN / 128];
#pragma unroll
  for (int q = 0; q < NA; ++q) qa[q].init(args.lda, args.M - m0 - 128 * q, wave, lane);
#pragma unroll
  for (int q = 0; q < NQ - NA; ++q) {
    if (GLU && LB == KC) qb[q].init_pairs(args.ldb, args.N - n0 - 64 * q, wave, lane);
    else if (GLU) qm[q].init_pairs(args.ldb, args.N - n0 - 64 * q, args.N, wave, lane);
    else if (LB == KC) qb[q].init(args.ldb, args.N - n0 - 128 * q, wave, lane);
    else qm[q].init(args.ldb, args.N - n0 - 128 * q, wave, lane);
  }

  auto slot = [&](int r, int q) -> char* { return smem + ((SPS * r + q) % NSLOT) * SLOT; };
  // Instruction i of this wave's share of quarter q of K step `step` (r = step % P).
  // Paired launches: steps nk .. 2 nk - 1 are product 1's steps 0 .. nk - 1.
  auto load = [&](int step, int r, int q, int i) {
    if (q >= NQ) return;
    const bool second = PAIR && step >= nk;
    const int k = k_begin + (second ? step - nk : step) * BK;
    const uint16_t* pa = second ? args_in.a_arr[1] : args.a;
    const uint16_t* pb = second ? args_in.b_arr[1] : args.b;
    char* dst = slot(r, q);
    if (q < NA) {
      qa[q].issue(make_rsrc(pa + (int64_t)(m0 + 128 * q) * args.lda + k), dst, k_end - k, wave, i);
    } else if (GLU && LB == KC) {
      qb[q - NA].issue(make_rsrc(pb + (int64_t)(n0 + 64 * (q - NA) + ((i & 1) ? args.N : 0)) * args.ldb + k), dst, k_end - k, wave, i);
    } else if (GLU) {
      qm[q - NA].issue(make_rsrc(pb + (int64_t)k * args.ldb + n0 + 64 * (q - NA)), dst, k_end - k, wave, i);
    } else if (LB == KC) {
      qb[q - NA].issue(make_rsrc(pb + (int64_t)(n0 + 128 * (q - NA)) * args.ldb + k), dst, k_end - k, wave, i);
    } else {
      qm[q - NA].issue(make_rsrc(pb + (int64_t)k * args.ldb + n0 + 128 * (q - NA)), dst, k_end - k, wave, i);
    }
  };

  f32x4_t acc[FI][FJ];
  f32x4_t acc2[PAIR ? FI : 1][PAIR ? FJ : 1];  // product 1's (paired launches)
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // (acc2 is cleared where product 1 starts, so that it holds no registers before.)

  if constexpr (F8 == 0) {
  bf16x8_t fa[FI], fb[2][FJ];
  // K-contiguous fragment f (rows 16f .. +15 of a 128-row quarter) in sub-step kk:
  // lane l reads row 16f + l % 16, 16-byte chunk 4kk + l / 16, at lane_kc[kk] + 2048 f.
  uint32_t lane_kc[2], lane_mc[FJ];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) lane_kc[kk] = tile16_off(lane & 15, 4 * kk + (lane >> 4));
  const int wcol = BN == 256 ? 0 : 64 * wn;  // the wave's first column inside its B quarter
#pragma unroll
  for (int j = 0; j < FJ; ++j) lane_mc[j] = mc16_lane_off(wcol + 16 * j, lane);
  // A fragment f of the wave: rows 16 f of its quarter (BM = 256: quarter wm),
  // or of its half of the one quarter (BM = 128: rows 64 wm + 16 f).
  auto read_a = [&](int r, int kk, int f) {
    const char* ta = BM == 256 ? slot(r, wm) + 2048 * f : slot(r, 0) + 2048 * (4 * wm + f);
    fa[f] = *reinterpret_cast<const bf16x8_t*>(ta + lane_kc[kk]);
  };
  auto read_b = [&](int buf, int r, int kk, int j) {
    const char* tb = slot(r, BN == 256 ? NA + wn : NA);
    if (LB == KC) {
      const int f = (BN == 256 ? 0 : 4 * wn) + j;  // 16-row block of the B quarter
      fb[buf][j] = *reinterpret_cast<const bf16x8_t*>(tb + lane_kc[kk] + 2048 * f);
    } else {
      const char* p = tb + lane_mc[j] + 8192 * kk;
      const i16x4_t lo = ds_read_tr(p), hi = ds_read_tr(p + 1024);
      const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      fb[buf][j] = __builtin_bit_cast(bf16x8_t, v);
    }
  };
  constexpr int NB = LB == KC ? FJ : 2 * FJ;  // LDS read instructions for the B fragments
  // acc += A B for one 16 x 16 block, the B fragment as the first operand.  Inline
  // assembly ties the accumulator to one AGPR quadruple for the whole K loop (the
  // builtin's results were moved between registers every iteration at this
  // register pressure).  The compiler still waits for the LDS reads that produce
  // the operands; the accumulators are next read by the epilogue, after explicit
  // wait states.
  auto mfma16 = [](f32x4_t& c, const bf16x8_t& b, const bf16x8_t& a) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
  };

  // One sub-step: the MFMAs on fa and fb[cur], row by row; with `reads`, the next
  // sub-step's fragments (ring position rn, sub-step kn): B into fb[1 - cur] during
  // row 0, A fragment f right after row f's MFMAs (its old value has then fed its
  // last MFMA).  Load n of the sub-step's NL goes after MFMA 1 (and FJ/2 + 1 for a
  // second) of row n * FI / NL.  Every MFMA with the reads and loads placed after it
  // is its own scheduling region, so the order is exactly this one.
  auto sub_step = [&](auto& C, int cur, bool reads, int rn, int kn, auto nl, auto&& issue_load) {
    constexpr int NL = decltype(nl)::value;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      int n_row = 0, n_first = 0;  // loads of this row and the first one's index
#pragma unroll
      for (int n = NL - 1; n >= 0; --n)
        if (n * FI / NL == i) {
          ++n_row;
          n_first = n;
        }
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        mfma16(C[i][j], fb[cur][j], fa[i]);
        if (reads && i == 0) {
#pragma unroll
          for (int u = 0; u < NB / FJ; ++u) {
            const int jb = j * (NB / FJ) + u;  // B read jb: fragment jb / (NB / FJ), half jb % (NB / FJ)
            if (NB == FJ || u == NB / FJ - 1) read_b(1 - cur, rn, kn, jb / (NB / FJ));
          }
        }
        if (j == 1 && n_row >= 1) issue_load(n_first);
        if (j == FJ / 2 + 1 && n_row >= 2) issue_load(n_first + 1);
        if (j == FJ - 1 && reads) read_a(rn, kn, i);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  auto vm_wait = [&](auto n) {
    constexpr int N = decltype(n)::value;
    static_assert(N >= 0 && N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  };
  using L0 = std::integral_constant<int, 0>;
  constexpr int HALF_LOADS = 4 * QS0;          // sub-step 0's quarters: 4 instructions each
  constexpr int TAIL_LOADS = 4 * (NQ - QS0);    // sub-step 1's
  constexpr int STEP_LOADS = HALF_LOADS + TAIL_LOADS;
  static_assert((D - 1) * STEP_LOADS < 64, "vmcnt");

  if (nk_all > 0) {
    // Prologue: steps 0 .. D-1 (as many as there are); wait for step 0.
#pragma unroll
    for (int st = 0; st < D; ++st)
      if (st < nk_all) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) load(st, st, q, i);
      }
    if (D >= 4 && nk_all >= 4) vm_wait(std::integral_constant<int, (D >= 4 ? 3 : 0) * STEP_LOADS>{});
    else if (D >= 3 && nk_all >= 3) vm_wait(std::integral_constant<int, (D >= 3 ? 2 : 0) * STEP_LOADS>{});
    else if (nk_all >= 2) vm_wait(std::integral_constant<int, STEP_LOADS>{});
    else vm_wait(L0{});
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < FJ; ++j) read_b(0, 0, 0, j);
#pragma unroll
    for (int f = 0; f < FI; ++f) read_a(0, 0, f);

    // K step k with LEFT = min(D, steps after it) known at compile time; r = k % P;
    // C the accumulator set of the step's product.
    auto k_step = [&](int k, auto left, int r, auto& C) {
      constexpr int LEFT = decltype(left)::value;
      const int r1 = r == P - 1 ? 0 : r + 1, rd = (r + D) % P;
      // sub-step 0: reads sub-step 1 of this step; loads the quarters of step k+D
      // whose slots step k does not use
      sub_step(C, 0, true, r, 1, std::integral_constant<int, LEFT >= D ? HALF_LOADS : 0>{},
               [&](int n) { load(k + D, rd, n >> 2, n & 3); });
      if constexpr (LEFT >= 1) {
        // Step k+1 has landed once at most the loads issued after its own are
        // in flight: whole steps k+2 .. k+D-1 and the part of step k+D just issued.
        constexpr int WHOLE = LEFT - 1 < D - 2 ? LEFT - 1 : D - 2;
        constexpr int AFTER = STEP_LOADS * (WHOLE > 0 ? WHOLE : 0) + (LEFT >= D ? HALF_LOADS : 0);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): sub-step 1's fragments are in registers
        vm_wait(std::integral_constant<int, AFTER>{});
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      // sub-step 1: reads sub-step 0 of step k+1; loads the rest of step k+D (for
      // 256-row tiles into step k's first slots)
      sub_step(C, 1, LEFT >= 1, r1, 0, std::integral_constant<int, LEFT >= D ? TAIL_LOADS : 0>{},
               [&](int n) { load(k + D, rd, QS0 + (n >> 2), n & 3); });
    };
    using Full = std::integral_constant<int, D>;
    int k = 0;
    if constexpr (PAIR) {
      // Product 0: steps 0 .. nk - 1 into acc, each with D or more steps after it
      // (the host pairs products of at least D K steps).
      for (; k + P <= nk; k += P) {
#pragma unroll
        for (int u = 0; u < P; ++u) k_step(k + u, Full{}, u, acc);
      }
      for (; k < nk; ++k) k_step(k, Full{}, k % P, acc);
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc2[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // The rest (product 1's steps into acc2 for paired launches), the last D
    // steps (or all of them, if fewer) each with its own LEFT.
    auto rest = [&](auto& C) {
      if constexpr (PAIR) {
        // Whole ring periods with the ring position known at compile time (both
        // accumulator sets are live here, and run-time positions cost registers);
        // the steps before nk and from the tail on are skipped.
        const int stop = nk_all - D;
        for (int k0 = nk - nk % P; k0 < stop; k0 += P) {
#pragma unroll
          for (int u = 0; u < P; ++u)
            if (k0 + u >= nk && k0 + u < stop) k_step(k0 + u, Full{}, u, C);
        }
      } else {
        for (; k + P + D <= nk_all; k += P) {  // steps k .. k+P-1, each with D more after it
#pragma unroll
          for (int u = 0; u < P; ++u) k_step(k + u, Full{}, u, C);
        }
        for (; k + D < nk_all; ++k) k_step(k, Full{}, k % P, C);
      }
      auto tail = [&](auto jc) {
        constexpr int J = decltype(jc)::value;
        if constexpr (J < D) {
          if (nk_all >= J + 1) k_step(nk_all - 1 - J, std::integral_constant<int, J>{}, (nk_all - 1 - J) % P, C);
        }
      };
      tail(std::integral_constant<int, 3>{});
      tail(std::integral_constant<int, 2>{});
      tail(std::integral_constant<int, 1>{});
      tail(std::integral_constant<int, 0>{});
    };
    if constexpr (PAIR) rest(acc2);
    else rest(acc);
    vm_wait(L0{});
  }
  } else {
    // FP8 operands (formats FA of A, FB of B: 0 E4M3, 1 E5M2).  A K step holds 128
    // FP8 values per row, the bytes of a bf16 step, so the ring, the loads and the
    // slot schedule are those above.  Each 16 x 16 block takes one
    // v_mfma_scale_f32_16x16x128_f8f6f4 per step (unit block scales; the tensors'
    // scales multiply the accumulators in the epilogue), on fragments of 32
    // bytes per lane: the two 16-byte fragments of a row that the bf16 sub-steps
    // read, in the same order for A and B (the instruction pairs the K positions
    // of its two operands lane by lane, so any common order is the same sum).
    // A step runs in two halves of FI/2 rows each, split by the mid-step wait and
    // barrier.  Half 0 reads A rows FI/2.. of this step after its rows; half 1
    // reads A rows 0..FI/2-1 of step k+1 after its rows, and B fragment j of step
    // k+1 right after the last MFMA that uses this step's fragment j.
    constexpr int FA = (F8 - 1) & 1, FB = (F8 - 1) >> 1, HR = FI / 2;
    typedef int i32x8_t __attribute__((ext_vector_type(8)));
    i32x8_t fa8[FI], fb8[FJ];
    uint32_t lane_kc[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) lane_kc[kk] = tile16_off(lane & 15, 4 * kk + (lane >> 4));
    auto frag8 = [&](const char* base) -> i32x8_t {
      const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(base + lane_kc[0]);
      const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(base + lane_kc[1]);
      return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };
    auto read_a8 = [&](int r, int f) {
      fa8[f] = frag8(BM == 256 ? slot(r, wm) + 2048 * f : slot(r, 0) + 2048 * (4 * wm + f));
    };
    auto read_b8 = [&](int r, int j) {
      fb8[j] = frag8(slot(r, BN == 256 ? NA + wn : NA) + 2048 * ((BN == 256 ? 0 : 4 * wn) + j));
    };
    const int unit_scale = 127;  // E8M0 block scale 2^0
    auto mfma8 = [&](f32x4_t& c, const i32x8_t& b, const i32x8_t& a) {
      if constexpr (FB == 0 && FA == 0)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel_hi:[0,0,0]"
                     : "+a"(c) : "v"(b), "v"(a), "v"(unit_scale));
      else if constexpr (FB == 1 && FA == 0)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel_hi:[0,0,0] cbsz:1"
                     : "+a"(c) : "v"(b), "v"(a), "v"(unit_scale));
      else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel_hi:[0,0,0] blgp:1"
                     : "+a"(c) : "v"(b), "v"(a), "v"(unit_scale));
    };
    auto vm_wait = [&](auto n) {
      constexpr int N = decltype(n)::value;
      static_assert(N >= 0 && N < 64, "vmcnt");
      __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
    };
    using L0 = std::integral_constant<int, 0>;
    constexpr int HALF_LOADS = 4 * QS0, TAIL_LOADS = 4 * (NQ - QS0), STEP_LOADS = HALF_LOADS + TAIL_LOADS;
    static_assert((D - 1) * STEP_LOADS < 64, "vmcnt");

    // Half h of a step at ring position r: rows h HR .. h HR + HR - 1.  With
    // `reads` (half 1 only), the next step's fragments come from ring position rn.
    auto half8 = [&](int h, int r, bool reads, int rn, auto nl, auto&& issue_load) {
      constexpr int NL = decltype(nl)::value;
#pragma unroll
      for (int ii = 0; ii < HR; ++ii) {
        const int i = h * HR + ii;
        int n_row = 0, n_first = 0;
#pragma unroll
        for (int n = NL - 1; n >= 0; --n)
          if (n * HR / NL == ii) {
            ++n_row;
            n_first = n;
          }
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          mfma8(acc[i][j], fb8[j], fa8[i]);
          if (h == 1 && reads && ii == HR - 1) read_b8(rn, j);
          if (j == 1 && n_row >= 1) issue_load(n_first);
          if (j == FJ / 2 + 1 && n_row >= 2) issue_load(n_first + 1);
          if (j == FJ - 1) {
            if (h == 0) read_a8(r, i + HR);
            else if (reads) read_a8(rn, i - HR);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };

    if (nk > 0) {
#pragma unroll
      for (int st = 0; st < D; ++st)
        if (st < nk) {
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) load(st, st, q, i);
        }
      if (D >= 4 && nk >= 4) vm_wait(std::integral_constant<int, (D >= 4 ? 3 : 0) * STEP_LOADS>{});
      else if (D >= 3 && nk >= 3) vm_wait(std::integral_constant<int, (D >= 3 ? 2 : 0) * STEP_LOADS>{});
      else if (nk >= 2) vm_wait(std::integral_constant<int, STEP_LOADS>{});
      else vm_wait(L0{});
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < FJ; ++j) read_b8(0, j);
#pragma unroll
      for (int f = 0; f < HR; ++f) read_a8(0, f);

      auto k_step8 = [&](int k, auto left, int r) {
        constexpr int LEFT = decltype(left)::value;
        const int r1 = r == P - 1 ? 0 : r + 1, rd = (r + D) % P;
        half8(0, r, false, r1, std::integral_constant<int, LEFT >= D ? HALF_LOADS : 0>{},
              [&](int n) { load(k + D, rd, n >> 2, n & 3); });
        if constexpr (LEFT >= 1) {
          constexpr int WHOLE = LEFT - 1 < D - 2 ? LEFT - 1 : D - 2;
          constexpr int AFTER = STEP_LOADS * (WHOLE > 0 ? WHOLE : 0) + (LEFT >= D ? HALF_LOADS : 0);
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): half 1's A fragments are in registers
          vm_wait(std::integral_constant<int, AFTER>{});
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        half8(1, r, LEFT >= 1, r1, std::integral_constant<int, LEFT >= D ? TAIL_LOADS : 0>{},
              [&](int n) { load(k + D, rd, QS0 + (n >> 2), n & 3); });
      };
      using Full = std::integral_constant<int, D>;
      int k = 0;
      for (; k + P + D <= nk; k += P) {
#pragma unroll
        for (int u = 0; u < P; ++u) k_step8(k + u, Full{}, u);
      }
      for (; k + D < nk; ++k) k_step8(k, Full{}, k % P);
      auto tail = [&](auto jc) {
        constexpr int J = decltype(jc)::value;
        if constexpr (J < D) {
          if (nk >= J + 1) k_step8(nk - 1 - J, std::integral_constant<int, J>{}, (nk - 1 - J) % P);
        }
      };
      tail(std::integral_constant<int, 3>{});
      tail(std::integral_constant<int, 2>{});
      tail(std::integral_constant<int, 1>{});
      tail(std::integral_constant<int, 0>{});
      vm_wait(L0{});
    }
  }
  // The last MFMAs' results are read below; 32 wait states cover the longest
  // write-to-read distance of a 16 x 16 x 32 MFMA (issued as inline assembly, so
  // the compiler does not insert them).
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __syncthreads();  // every wave is done with the operand slots

  // Epilogue, one 64 x 64 chunk of the wave's sub-tile at a time (FI / 4 chunks
  // tall, FJ / 4 wide), staged in the wave's own 16 KiB of LDS.  Block (i, j)
  // register e holds C[16i + lane%16][16j + 4 (lane/16) + e] of the wave's
  // sub-tile.
  // FP8: the product of the two tensors' scales (unit for bf16 operands).
  // FP8: the two operands' amax slots in one load, one word per lane (lanes 0-15
  // the words of A's slot, 16-31 B's); the epilogue takes the max over each
  // 16-lane group (lane 0 then holds A's amax, lane 16 B's) once its first loads
  // are issued.
  static_assert(2 * AMAX_SUB <= 64 && (AMAX_SUB & (AMAX_SUB - 1)) == 0, "two slots' words fit one wave");
  uint32_t amax_word = 0;
  if (F8 != 0 && lane < 2 * AMAX_SUB)
    amax_word = (lane < AMAX_SUB ? args.amax_a : args.amax_b)[(lane & (AMAX_SUB - 1)) * AMAX_SUB_STRIDE];
  auto scales = [&]() {
#pragma unroll
    for (int off = AMAX_SUB / 2; off > 0; off >>= 1)
      amax_word = max(amax_word, (uint32_t)__shfl_xor((int)amax_word, off, 64));
    const float amax_a = __builtin_bit_cast(float, __builtin_amdgcn_readlane((int)amax_word, 0));
    const float amax_b = __builtin_bit_cast(float, __builtin_amdgcn_readlane((int)amax_word, AMAX_SUB));
    return fp8_scale_of(amax_a, fp8_fmax((F8 - 1) & 1)) * fp8_scale_of(amax_b, fp8_fmax((F8 - 1) >> 1));
  };
  store_staged<EPI, (FI / 4) * (FJ / 4), F8 != 0>(
      [&](int ch, float sc) {
        const int h = ch % (FI / 4), hc = ch / (FI / 4);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const int r = 16 * ii + (lane & 15), c = 4 * jj + (lane >> 4);
            f32x4_t v = acc[4 * h + ii][4 * hc + jj];
            if constexpr (F8 != 0) v = v * sc;
            *reinterpret_cast<f32x4_t*>(smem + wave * (64 * ROW_B) + r * ROW_B + ((c ^ (r & 15)) << 4)) = v;
          }
      },
      scales, args, smem + wave * (64 * ROW_B), m0 + (BM / 2) * wm, n0 + (GLU ? BN / 4 : BN / 2) * wn, FI / 4, split, lane,
      // paired launches: product 1's chunk in the LDS above the four waves' first regions
      [&](int ch) {
        if constexpr (PAIR) {
          const int h = ch % (FI / 4), hc = ch / (FI / 4);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const int r = 16 * ii + (lane & 15), c = 4 * jj + (lane >> 4);
              *reinterpret_cast<f32x4_t*>(smem + (4 + wave) * (64 * ROW_B) + r * ROW_B + ((c ^ (r & 15)) << 4)) =
                  acc2[4 * h + ii][4 * hc + jj];
            }
        }
      },
      smem + (4 + wave) * (64 * ROW_B));

// Host-side audit of the loads into LDS that only the linears with an epilogue make (built and run by
// tests/test_block_dma_audit.py; no GPU involved), with the checks of dma_audit.hip: the fp8r tiles' hand-ordered loop at
// any K, and the nvfp4 tiles at K % 256 != 0, whose block scales go through registers.
#define main audit_of_the_plain_linears
#include "dma_audit.hip"
#undef main

namespace {

// ---- fp8r (gemm_fp8_epilogue.hip): stages 0 .. nk - 1; all but the last with the lane offsets of stage 0, the last one
// with its own
template <int BM, int BN>
void audit_fp8_any_k(int M, int N, int K) {
  using C = Fp8Cfg<BM, BN, 2>;
  char cfg[96];
  std::snprintf(cfg, sizeof cfg, "fp8 any K %dx%d, %dx%dx%d", BM, BN, M, N, K);
  const int nk = (K + C::KSTAGE - 1) / C::KSTAGE, LA = C::RA::MIN_PER_WAVE;
  auto load = [&](int i, int ld, int lane, int kb) {
    return i < LA ? region_load<typename C::RA>(ld, lane, K, kb, kb, K)
                  : region_load<typename C::RB>(ld, lane, K, kb, kb, K);
  };
  for (int tm : edge_tiles(M, BM))
    for (int tn : edge_tiles(N, BN)) {
      const int rows_x = std::min(BM, M - tm * BM), rows_w = std::min(BN, N - tn * BN);
      for (int kt = 0; kt < nk; ++kt) {
        const int kb = kt * C::KSTAGE, slot = (kt % 2) * C::STAGE;
        std::vector<char> put(C::STAGE / 16, 0);
        for (int wave = 0; wave < 4; ++wave)
          for (int i = 0; i < C::LOADS_MIN; ++i) {
            const int ld = wave + 4 * (i < LA ? i : i - LA), rows = i < LA ? rows_w : rows_x;
            for (int lane = 0; lane < 64; ++lane) {
              DmaAddr d = load(i, ld, lane, kb);
              if (kt < nk - 1) d.voff = load(i, ld, lane, 0).voff;
              const int chunk = swz_chunk<128>(ld * C::RA::RPL + lane / C::RA::C, lane % C::RA::C);
              check_lane(cfg, d, slot + (i < LA ? 0 : C::A_BYTES), 16, C::LDS, slot, slot + C::STAGE,
                         (uint32_t)(rows * K), rows, K, K, kb + 16 * chunk < K);
              ++put[((i < LA ? 0 : C::A_BYTES) + d.lds) / 16];
            }
          }
        for (size_t c = 0; c < put.size(); ++c)
          if (put[c] != 1) fail(cfg, "a chunk of a stage is not written once", (long)c, put[c], kt, 0);
      }
    }
  std::printf("ok %s\n", cfg);
}

// ---- nvfp4 (gemm_w4a4_any_epilogue.hip): codes by LDS DMA (stage 1 also where there is none), block scales through
// registers
template <int BM, int BN>
void audit_w4a4_any_k(int M, int N, int K) {
  using C = W4Cfg<BM, BN>;
  char cfg[96];
  std::snprintf(cfg, sizeof cfg, "w4a4 any K %dx%d, %dx%dx%d", BM, BN, M, N, K);
  const int nk = (K + C::KSTAGE - 1) / C::KSTAGE, kp = K / 2, ks = K / 16;
  for (int tm : edge_tiles(M, BM))
    for (int tn : edge_tiles(N, BN)) {
      const int m0 = tm * BM, n0 = tn * BN, rows_x = std::min(BM, M - m0), rows_w = std::min(BN, N - n0);
      for (int kt = 0; kt < std::max(nk, 2); ++kt) {
        const int kb = kt * C::KSTAGE, slot = (kt & 1) * C::STAGE;
        audit_region<typename C::RA>(cfg, slot + C::A_OFF, C::LDS, slot, slot + C::STAGE, (uint32_t)(rows_w * kp),
                                     rows_w, kp, kp, kp, kb >> 1, kb, K, 32, true);
        audit_region<typename C::RB>(cfg, slot + C::B_OFF, C::LDS, slot, slot + C::STAGE, (uint32_t)(rows_x * kp),
                                     rows_x, kp, kp, kp, kb >> 1, kb, K, 32, true);
        std::vector<char> put(C::STAGE / 16, 0);
        for (int r = 0; r < (BM + BN + 255) / 256 * 256; ++r) {  // (256 threads, whole steps)
          ++g_lanes;
          const ScaleRowLoad l = scale_row_load<BM, BN>(r, kt, m0, n0, M, N, K);
          if (l.lds != scale_row_load<BM, BN>(r, 0, 0, 0, 0, 0, 0).lds) fail(cfg, "LDS place of scales moves", r, l.lds, kt, 0);
          if (r >= BM + BN) {
            if (l.left != 0 || l.lds >= 0) fail(cfg, "scales of a row past the tile", r, l.left, l.lds, 0);
            continue;
          }
          const bool w = r < BN;
          const int row = w ? n0 + r : m0 + r - BN, rows = w ? N : M, want = row < rows ? std::max(0, ks - kt * 16) : 0;
          if (l.w != w) fail(cfg, "scales of the other operand", r, l.w, 0, 0);
          if (l.left != want) fail(cfg, "scales left of a row", r, l.left, want, kt);
          if (l.left & 1) fail(cfg, "half of two scales", r, l.left, 0, 0);
          const int bytes = std::min(l.left, 16);
          if (bytes > 0) {
            if (l.from & 1) fail(cfg, "odd address of scales", r, (long)l.from, 0, 0);
            if (l.from / ks != row || (l.from + bytes - 1) / ks != row) fail(cfg, "scales of another row", r, (long)l.from, row, ks);
            if (l.from % ks != kt * 16) fail(cfg, "scales of another stage", r, (long)l.from, kt, ks);
            if (l.from < 0 || l.from + bytes > (int64_t)rows * ks) fail(cfg, "scales outside the operand", r, (long)l.from, bytes, rows);
          }
          const int at = (w ? C::SA_OFF + 16 * r : C::SB_OFF + 16 * (r - BN));
          if (l.lds != at || at + 16 > C::STAGE || slot + at + 16 > C::LDS) fail(cfg, "LDS place of scales", r, l.lds, at, 0);
          ++put[l.lds / 16];
        }
        for (int c = C::SA_OFF / 16; c < C::STAGE / 16; ++c)
          if (put[c] != 1) fail(cfg, "scales of a row are not written once", c, put[c], kt, 0);
      }
    }
  std::printf("ok %s\n", cfg);
}

}  // namespace

int main() {
  // one stage, two and more, whole and partial; ragged rows; the largest K of a large tile, and one of odd depth
  for (int K : {32, 96, 128, 160, 224, 256, 288, 544, 1056, 1184, 6048, 20512, 65536 + 32})
    for (auto& s : {std::pair<int, int>{64, 64}, {70, 90}, {777, 1234}, {1030, 2049}, {4500, 6100}}) {
      audit_fp8_any_k<128, 128>(s.first, s.second, K);
      audit_fp8_any_k<256, 192>(s.first, s.second, K);
      audit_fp8_any_k<256, 256>(s.first, s.second, K);
      audit_fp8<64, 64, 4>(s.first, s.second, K);   // the general loop of the smaller tiles
      audit_fp8<64, 128, 4>(s.first, s.second, K);
      if (K % 256 != 0) {
        audit_w4a4_any_k<64, 64>(s.first, s.second, K);
        audit_w4a4_any_k<128, 128>(s.first, s.second, K);
        audit_w4a4_any_k<256, 192>(s.first, s.second, K);
      } else {
        audit_w4a4<64, 64>(s.first, s.second, K);
        audit_w4a4<64, 128>(s.first, s.second, K);
        audit_w4a4<128, 128>(s.first, s.second, K);
        audit_w4a4<256, 192>(s.first, s.second, K);
        audit_w4a4<256, 256>(s.first, s.second, K);
      }
    }
  audit_fp8_any_k<256, 256>(70, 300, (1 << 20) - 32);  // the largest K that a linear takes with a partial last stage
  audit_w4a4_any_k<256, 192>(70, 300, (1 << 20) - 32);
  std::printf("all loads of the linears with an epilogue in bounds: %ld lanes checked\n", g_lanes);
  return 0;
}

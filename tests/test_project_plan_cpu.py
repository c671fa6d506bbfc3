"""Plans of the projection of few rows (csrc/project_plan.h), swept on the host over its shapes.

An SM has 228 KB of shared memory, of which a CTA takes 1 KB beside its own, and 512 columns of
tensor memory, which a CTA of project_kernel asks for whole and waits for without a limit.  So no two
CTAs that wait for one another (those of a cluster) may be placed on one SM, whichever streams they
come from: each asks for more than the half of its shared memory, and for more than a clustered CTA of
gemv_mma.cu leaves (73 KB at least).  Neither may one that is of no cluster wait between two of those,
in front of the other's turn.
"""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SWEEP = r"""
#include <cstdio>
#include "project_plan.h"
using namespace tts;
static int bad = 0;
static void expect(bool ok, const char* what, int rows, int n, int k, int es, int rm, int tc, const Plan& q) {
  if (ok) return;
  if (++bad <= 20)
    printf("%s: rows %d n %d k %d es %d rm %d tc %d: nb %d split %d stages %d ch %d groups %d smem %d\n", what, rows, n, k, es,
           rm, tc, q.nb, q.split, q.stages, q.ch, q.groups, q.smem);
}
int main() {
  const int kSm = 228 * 1024, kStatic = 3328, kOwn = 1024, n_sm = 152;
  const int budget = kSm - kOwn - kStatic;
  const int rows[] = {1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 80, 96, 100, 127, 128, 129, 144, 159, 160, 161, 176, 191, 192,
                      193, 200, 224, 255, 256, 257, 300, 319, 320, 321, 480, 500, 1000, 1025, 4096, 20000, 1 << 20};
  const int ns[] = {1, 7, 127, 128, 129, 256, 520, 1000, 2048, 4096, 6144, 9700, 12288, 16384, 19456, 24000, 1 << 20};
  const int ks[] = {16, 32, 64, 80, 96, 128, 144, 192, 208, 256, 384, 512, 640, 1024, 2048, 2064, 5120, 12288, 65536};
  const int rms[] = {0, 8, 16, 24, 32, 40, 64, 72, 80, 96, 104, 112, 128};
  long plans = 0, clusters = 0, single = 0;
  for (int r : rows) for (int n : ns) for (int k : ks) for (int es = 1; es <= 2; ++es) for (int rm : rms)
    for (int tc = 0; tc <= (rm > 0 && r >= 128); ++tc) {
      Plan q;
      const int threads = max_threads(rm > 64);
      const bool fits = plan_rows(q, r, n, k, es, rm, tc, budget, n_sm, [&](int split, int smem) {
        int per = kSm / (smem + kStatic + kOwn);
        if (per > 2048 / threads) per = 2048 / threads;
        return n_sm * per / split;
      });
      ++plans;
      expect(fits, "does not fit", r, n, k, es, rm, tc, q);
      if (!fits) continue;
      const int chunk = kWChunk + q.nb * kRowBytes, per = (q.nb + q.split - 1) / q.split;
      expect(q.nb % 16 == 0 && q.nb >= 16 && q.nb <= 256, "rows of a tile", r, n, k, es, rm, tc, q);
      expect(static_cast<int64_t>(q.n_rt) * q.nb >= r && (q.n_rt - 1) * static_cast<int64_t>(q.nb) < r, "tiles", r, n, k, es, rm, tc, q);
      expect(q.n_acc * q.nbr + (rm > 0 ? q.nbr : 0) <= 512, "tensor memory", r, n, k, es, rm, tc, q);
      expect(q.stages >= 1 && q.stages <= kMaxStages && q.stages * q.ch * chunk <= q.v_off, "ring", r, n, k, es, rm, tc, q);
      expect(per * rm * 4 <= q.b_off - q.v_off, "v", r, n, k, es, rm, tc, q);
      expect(128 * q.groups + 64 <= threads && (rm == 0 || per >= q.groups), "groups", r, n, k, es, rm, tc, q);
      expect(2 * (q.smem + kStatic + kOwn) > kSm, "two CTAs on an SM", r, n, k, es, rm, tc, q);
      expect(q.smem + kStatic + kOwn + 73 * 1024 > kSm, "beside a CTA of gemv_mma", r, n, k, es, rm, tc, q);
      if (q.split > 1) {
        ++clusters;
        expect(q.nb * kRedLd * 4 <= q.v_off, "partial sums", r, n, k, es, rm, tc, q);
      }
      single += q.stages == 1 && q.n_chunks > 1;
    }
  printf("%ld plans, %ld in clusters, %ld with one stage, %d bad\n", plans, clusters, single, bad);
  return bad != 0;
}
"""


@pytest.fixture(scope="module")
def sweep(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    src, exe = at / "sweep.cpp", at / "sweep"
    src.write_text(SWEEP)
    csrc = os.path.join(ROOT, "autoregressive_codebook_tts_gb300", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_every_plan_fits_and_no_cta_meets_one_that_waits_for_a_cluster(sweep):
    assert sweep.returncode == 0, sweep.stdout

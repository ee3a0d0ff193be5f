"""Tensor memory of kernels that share an SM, without a GPU: whatever they are and
whatever the rank, the blocks that an SM has shared memory for never leave a
cluster's block waiting for columns that other clusters' blocks hold."""
import itertools
import subprocess

import pytest

SM, COLUMNS, SYSTEM = 228 << 10, 512, 1 << 10  # an SM's shared memory and TMEM columns; the system's part of a block

# (name, rank or tokens, columns, bytes of shared memory, in a cluster) of every launch, static arrays taken as `fixed`
PROGRAM = r"""
#include <cstdio>
#include "tmem.h"
using namespace rgs;
static void put(const char* name, int n, uint32_t columns, size_t dynamic, size_t fixed, int clusters) {
  const size_t bytes = dynamic + fixed + kBlockSmem;
  std::printf("%s %d %u %zu %d %d\n", name, n, columns, bytes, clusters, (int)tmem_safe(columns, bytes, clusters));
}
int main(int, char** argv) {
  const size_t fixed = (size_t)atoi(argv[1]);
  for (int r = 1; r <= kMaxRank; ++r) {
    const int n_pad = (r + 15) / 16 * 16;
    const uint32_t a = 128 * 64 * 2, b_proj = n_pad * 64 * 2, b_acc = (n_pad + 63) / 64 * 64 * 64 * 2;
    const SkinnySizes s[3] = {skinny_sizes(n_pad, a, b_proj, 2, fixed), skinny_sizes(n_pad, a, b_acc, 1, fixed),
                              skinny_sizes(n_pad, a, b_acc, 2, fixed)};
    const char* names[3] = {"project", "accumulate", "accumulate_fp32xp"};
    for (int i = 0; i < 3; ++i) put(names[i], r, s[i].tmem_cols, s[i].smem, fixed, 1);
    const PersistentSizes p[3] = {project_sizes(n_pad, a, b_proj).p, accumulate_sizes(n_pad, b_acc, 1, 1),
                                  accumulate_sizes(n_pad, b_acc, 1, 2)};
    for (int i = 0; i < 3; ++i) {
      if (p[i].stages < 2) return 1;
      put("persistent", r, p[i].tmem_cols, p[i].smem, fixed, 0);
    }
    const GramSizes g = gram_sizes(r, fixed);
    for (int stages = 0; stages <= g.raw_stages; ++stages) put("gram", r, gtc_tmem_cols(r), gram_ring_smem(g, r, stages), fixed, 0);
    put("triangular", r, ttc_tmem_cols(r), ttc_smem_bytes(r), fixed, 0);
    const int ncols = n_pad <= 128 ? 128 : 64, kchunks = (n_pad + 63) / 64;
    const UpdateSizes u = update_sizes(kchunks, 2 * kchunks * 16384, 2 * ncols * 128, ncols / 64 * 16384, fixed);
    if (u.w_stages < 1) return 1;
    put("update", r, kTmemBufs * ncols, u.smem, fixed, 0);
  }
  for (int tokens : {16, 32, 64}) put("few", tokens, few_columns(tokens), few_smem(tokens, fixed), fixed, 1);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from rank_gradient_sketching_philox_gb300 import build_lib
    at = tmp_path_factory.mktemp("tmem")
    (at / "tmem.cu").write_text(PROGRAM)
    subprocess.run([build_lib._nvcc(), "-std=c++17", "-I", build_lib.INCLUDE, "-I", build_lib.CSRC, str(at / "tmem.cu"),
                    "-o", str(at / "tmem")], check=True, capture_output=True)
    return str(at / "tmem")


def launches(program, fixed):
    out = subprocess.run([program, str(fixed)], check=True, capture_output=True, text=True).stdout
    rows = [line.split() for line in out.splitlines()]
    return [(n, int(r), int(c), int(b), bool(int(k)), bool(int(safe))) for n, r, c, b, k, safe in rows]


def too_many(blocks):
    """Blocks (columns, bytes, in a cluster) that fit an SM, two or more of clusters among them, and want more columns
    than it has; None where there are no such."""
    kinds = sorted(set(blocks), key=lambda b: b[1])
    for n in range(2, SM // kinds[0][1] + 1):
        for mix in itertools.combinations_with_replacement(kinds, n):
            if (sum(b[1] for b in mix) <= SM and sum(b[0] for b in mix) > COLUMNS and sum(b[2] for b in mix) >= 2):
                return mix
    return None


def least(blocks):
    """Of the blocks with the same columns and kind, those with the least bytes: they fit wherever the others do."""
    by = {}
    for c, b, k in blocks:
        by[c, k] = min(b, by.get((c, k), SM))
    return [(c, b, k) for (c, k), b in by.items()]


@pytest.mark.parametrize("fixed", [0, 96, 736, 2208, 4096])
def test_no_mix_of_launches_wants_more_columns_than_there_are(program, fixed):
    rows = launches(program, fixed)
    assert {n for n, *_ in rows} == {"project", "accumulate", "accumulate_fp32xp", "persistent", "gram", "triangular", "update", "few"}
    for name, r, columns, size, clusters, safe in rows:
        assert safe and size <= SM, (name, r, columns, size)
    blocks = least([(c, b, k) for _, _, c, b, k, _ in rows] + [(512, 197632 + SYSTEM, True)])  # the pairs that take all of TMEM
    assert too_many(blocks) is None


def test_the_shares_leave_room_for_the_blocks_that_they_are_meant_for(program):
    """Four blocks of up to 16 tokens on an SM, two of the others in clusters, as many Gram blocks as TMEM has columns for."""
    for name, r, columns, size, clusters, _ in launches(program, 736):
        if name == "few":
            assert SM // size == COLUMNS // columns
        if name == "accumulate" and r <= 192:
            assert SM // size == 2, r
        if name == "gram":
            assert SM // size >= min(2, COLUMNS // columns), r


def test_a_mix_that_would_wait_is_found():
    """Accumulations at ranks 129 to 160 with 86176 bytes for their 256 columns, and products of up to 16 tokens with 58080
    for 128, as they once were: two of the first and one of the second want 640 columns."""
    mix = too_many([(256, 86176, True), (128, 58080, True)])
    assert mix is not None and sum(b[0] for b in mix) == 640
    assert too_many([(256, 116736, True), (128, 58368, True)]) is None
    assert too_many([(512, 116752, False), (128, 58368, True)]) is None
    assert too_many([(512, 116752, False), (128, 58080, True)]) is not None


def test_the_rule_refuses_what_is_too_small(tmp_path):
    from rank_gradient_sketching_philox_gb300 import build_lib
    (tmp_path / "rule.cu").write_text(r"""
#include "tmem.h"
using namespace rgs;
static_assert(!tmem_safe(256, 86176, true) && !tmem_safe(128, 58080, true) && !tmem_safe(256, 77936, false));
static_assert(tmem_safe(256, 116736, true) && tmem_safe(128, 58368, true) && tmem_safe(512, 116752, false));
static_assert(!tmem_safe(512, 116736, false) && !tmem_safe(512, 166000, true) && !tmem_safe(32, 40000, true));
static_assert(!tmem_safe(1024, 233472, true) && !tmem_safe(512, 233473, true) && tmem_safe(512, 198656, true));
int main() {}
""")
    subprocess.run([build_lib._nvcc(), "-std=c++17", "-I", build_lib.INCLUDE, "-I", build_lib.CSRC, "-c", str(tmp_path / "rule.cu"),
                    "-o", str(tmp_path / "rule.o")], check=True, capture_output=True)

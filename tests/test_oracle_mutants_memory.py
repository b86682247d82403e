"""Planted mistakes of the oracle stay within memory that is theirs (CPU only):
with fresh memory filled with a pattern they are caught, not killed."""
import os
import subprocess
import sys

import pytest

import oracle
from drafter_vocab_top_amd import workloads as W

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name", ["last_row_skipped", "layout_transposed"])
def test_planted_mistakes_read_no_stray_memory(name):
    """MALLOC_PERTURB_ (without glibc's per-thread caches) makes what a mistake reads of fresh memory a pattern: as
    a row id it would point gigabytes away."""
    env = {**os.environ, "MALLOC_PERTURB_": "165", "GLIBC_TUNABLES": "glibc.malloc.tcache_count=0"}
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "test_oracle_mutants.py", "-k", name],
                       cwd=HERE, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_an_alternative_build_gets_the_whole_square():
    """What lies behind the matrix of an alternative build is zero, up to the
    elements that rows and columns exchanged would reach."""
    V, C, ld = 5, 2, 6

    class Lib:
        def oracle_topk_cols(self, V, C, k, dtype, layout, ld, x, values, ids, nthreads):
            import ctypes
            self.seen = list((ctypes.c_uint16 * (V * ld)).from_address(x))
            return 0
    lib = Lib()
    x = W.random_matrix(1, V, C, W.BF16, W.COL, ld=ld)
    oracle.topk_cols(x, V, C, 1, oracle.BF16, oracle.COL_CONTIG, ld, lib=lib)
    flat = x.reshape(-1)
    assert lib.seen[:flat.size] == flat.tolist() and not any(lib.seen[flat.size:])

"""What can be seen of the kernels' sources without a GPU."""
import glob
import os

import speculative_decoding_verify_temp_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def test_no_uniform_branch_on_a_threads_own_predicate():
    # mbarrier.try_wait answers each thread; a .uni branch on an answer that differs within a warp is undefined
    files = glob.glob(os.path.join(CSRC, "*.cu*"))
    assert files
    for f in files:
        with open(f) as src:
            assert "bra.uni" not in src.read(), f

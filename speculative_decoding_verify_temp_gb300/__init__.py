"""GB300-native speculative-decoding verify-and-sample step.

The product is ``libtsverify.so`` (C ABI declared in ``include/ts_verify.h``, kernels
for sm_103a under ``csrc/``); ``tsverify`` is its thin ctypes binding and ``synth``
the seeded synthetic input generator shared by the tests and the benchmark.
"""
from . import tsverify  # noqa: F401
from .tsverify import (  # noqa: F401
    chain_spec_sampling,
    gather_logprobs,
    gumbel_max_sample,
    kv_append,
    kv_read,
    make_attention_workspace,
    make_workspace,
    softmax_temp,
    topk_topp_renorm,
    tree_spec_sampling,
    verify_chain_greedy,
    window_attention,
)

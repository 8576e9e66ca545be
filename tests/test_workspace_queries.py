"""Workspace queries on the CPU: for arguments that the call itself refuses a query returns 0 and the
process goes on.  The wrappers ask before the call checks, so a query that fails on them takes the
interpreter down.  Each query runs in a process of its own, which prints what it is about to ask."""
import subprocess
import sys

import pytest

ASK = """
import itertools, sys
import semi_structured_sparsity_amd as nm
query = getattr(nm.raw, {name!r})
for args in {cases!r}:
    print("asking", args, flush=True)
    assert query(*args) == 0, (args, query(*args))
print("answered", flush=True)
"""

# (K, Ns) that no product takes: patterns that do not exist, and widths without a whole group
REFUSED = [(64, 1), (64, 2), (64, 9), (64, -1), (64, 100), (1, -1), (4, 4), (4, 1), (14, 8), (1, 3), (63, 4), (72, 7), (0, 4), (-8, 4)]
TOKENS_ROWS = [(1, 8), (4, 8), (40, 300), (200, 4096), (2048, 4096)]


def _ask(name, cases):
    r = subprocess.run([sys.executable, "-c", ASK.format(name=name, cases=cases)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "answered" in r.stdout, (r.returncode, r.stdout[-200:], r.stderr[-400:])


@pytest.mark.parametrize("name,last", [("nm_spmm_workspace", (1, 2, 4)), ("nm_spmm_glu_workspace", (1, 2, 4)),
                                       ("nm_spmm_lowrank_workspace", (8, 256))])
def test_product_queries(name, last):
    _ask(name, [(M, K, R, Ns, x) for M, R in TOKENS_ROWS for K, Ns in REFUSED for x in last])


@pytest.mark.parametrize("name", ["nm_spmm_backward_workspace", "nm_spmm_glu_backward_workspace"])
def test_backward_queries(name):
    most = 1 << 21
    _ask(name, [(M, K, R, Ns) for M, R in TOKENS_ROWS for K, Ns in REFUSED] +
         [(1, most, 1 << 40, 8), (4, most, 1 << 40, 4), (33, 1 << 40, 8, 0), (most + 1, 64, 8, 0)])


def test_queries_of_what_the_calls_take_are_unchanged():
    """Sizes by formula: the lifted activation of a many-token product, the plain product's none."""
    import semi_structured_sparsity_amd as nm
    q = nm.raw.nm_spmm_workspace
    assert q(2048, 4096, 11008, 0, nm.NM_BF16) == 0
    for Ns, K in ((3, 768), (4, 1024), (5, 640), (8, 1024)):
        assert q(2048, K, 4096, Ns, nm.NM_BF16) >= 2048 * nm.lifted_width(K, Ns) * 2
        assert nm.raw.nm_spmm_glu_workspace(2048, K, 4096, Ns, nm.NM_BF16) >= 2048 * nm.lifted_width(K, Ns) * 2
        assert nm.raw.nm_spmm_lowrank_workspace(2048, K, 4096, Ns, 16) >= 2048 * nm.lifted_width(K, Ns) * 2
        assert nm.raw.nm_spmm_backward_workspace(2048, K, 4096, Ns) >= 2048 * (K + 2 * 4096) * 2


def test_wrapper_refuses_a_pattern_that_does_not_exist():
    """nm_spmm_glu(..., Ns=1) on CPU tensors reaches the query and then an error, in a process of its own."""
    code = """
import torch, semi_structured_sparsity_amd as nm
x, v = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 32), dtype=torch.bfloat16)
i = torch.zeros((8, 4), dtype=torch.int32)
for Ns in (1, -1):
    try:
        nm.nm_spmm_glu(x, v, i, v.clone(), i.clone(), Ns=Ns)
    except (ValueError, nm.NMError) as e:
        print("refused", type(e).__name__)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.count("refused") == 2, (r.returncode, r.stdout, r.stderr[-400:])

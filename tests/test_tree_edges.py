"""Draft-tree calls at the edges of their arguments (no GPU: refused, or nothing to do)."""

import pytest

from tests.test_tree_abi import ARG, CALLS, OK, L, call  # noqa: F401

PER_NODE = {"mla_tree_write": ("h", "token"),
            "mla_tree_absorb_q": ("q_nope", "q_rope", "token", "q_abs"),
            "mla_attend_tree": ("q_abs", "tree", "o_lat", "lse"),
            "mla_attend_weight": ("q_abs", "tree", "lse", "query_weight"),
            "mla_tree_accept": ("accept",)}


@pytest.mark.parametrize("name", PER_NODE)
def test_empty_per_node_tensors_may_be_null(L, name):  # noqa: F811
    """What torch passes for a tensor without elements; the other tensors are still needed."""
    none = dict.fromkeys(PER_NODE[name])
    assert call(L, name, n=0, **none) == OK
    assert call(L, name, n=1, **none) == ARG
    for k in {"window", "cache", "w_dkv", "w_kr", "w_uk", "weight_out", "ws"} & set(CALLS[name]):
        if (name, k) != ("mla_attend_tree", "ws"):
            assert call(L, name, n=0, **none, **{k: None}) == ARG, k

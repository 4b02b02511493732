"""Argument checks of the draft-tree and eviction calls (no GPU: refused before any launch)."""

import ctypes

import pytest

from latent_kv_cache_write_b200 import build, native
from synth import configs as C

FAKE, ODD, BYTE = 0x10000, 0x10008, 0x10001
OK, ARG, UNS, ALIGN, RANGE = (native.MLA_OK, native.MLA_ERR_ARG, native.MLA_ERR_UNSUPPORTED,
                              native.MLA_ERR_ALIGN, native.MLA_ERR_RANGE)


@pytest.fixture(scope="module")
def L():
    build.build()
    return native.lib()


def shape(**kw):
    s = native.make_shape(C.DECODE)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


CALLS = {
    # name: (argument names in order, defaults)
    "mla_tree_write": dict(h=FAKE, d_model=4096, n=4, window=FAKE, token=FAKE, w_dkv=FAKE,
                           w_kr=FAKE, cache=FAKE, position=FAKE),
    "mla_tree_absorb_q": dict(q_nope=FAKE, q_rope=FAKE, n=4, token=FAKE, w_uk=FAKE, q_abs=FAKE),
    "mla_attend_tree": dict(q_abs=FAKE, n=4, cache=FAKE, window=FAKE, tree=FAKE, scale=0.07,
                            o_lat=FAKE, lse=FAKE, ws=None, ws_bytes=0),
    "mla_attend_weight": dict(q_abs=FAKE, n=4, cache=FAKE, window=FAKE, tree=FAKE, scale=0.07,
                              lse=FAKE, query_weight=FAKE, weight_in=FAKE, weight_out=FAKE),
    "mla_tree_accept": dict(cache=FAKE, n=4, accept=FAKE, window=FAKE, weight=FAKE, position=FAKE,
                            ws=FAKE, ws_bytes=1 << 30),
    "mla_cache_evict": dict(cache=FAKE, keep=4, sink=0, recent=0, window=FAKE, weight=FAKE,
                            position=FAKE, ws=FAKE, ws_bytes=1 << 30),
}
OPTIONAL = {"mla_tree_write": {"position"}, "mla_attend_tree": {"tree", "lse", "ws"},
            "mla_attend_weight": {"tree", "query_weight", "weight_in"},
            "mla_tree_accept": {"weight", "position"}}
WIDE_ALIGN = {"h", "w_dkv", "w_kr", "cache", "q_nope", "q_rope", "w_uk", "q_abs", "o_lat"}


def call(L, name, s=None, **kw):
    args = dict(CALLS[name], **kw)
    s = s or shape()
    return getattr(L, name)(ctypes.byref(s), *args.values(), None)


@pytest.mark.parametrize("name", CALLS)
def test_pointers(L, name):
    for k, v in CALLS[name].items():
        if v != FAKE:
            continue
        if k not in OPTIONAL.get(name, ()):
            assert call(L, name, **{k: None}) == ARG, k
        if k not in ("tree", "accept"):
            assert call(L, name, **{k: BYTE}) == ALIGN, k
        if k in WIDE_ALIGN or k == "ws" or (k == "lse" and name == "mla_attend_tree"):
            assert call(L, name, **{k: ODD}) == ALIGN, k


@pytest.mark.parametrize("name", [n for n in CALLS if n != "mla_cache_evict"])
def test_node_counts(L, name):
    assert call(L, name, n=-1) == ARG
    assert call(L, name, n=8193) == RANGE                    # more nodes than slots
    assert call(L, name, n=0) == OK                            # nothing to do
    assert call(L, name, shape(batch=0)) == ARG
    assert call(L, name, shape(ring_slots=1 << 31)) == UNS


def test_sizes_beyond_32_bits(L):
    big = shape(batch=500, n_heads=128, ring_slots=60000)
    for name in ("mla_tree_absorb_q", "mla_attend_tree", "mla_attend_weight"):
        assert call(L, name, big, n=40000) == UNS, name
    tall = shape(batch=1, ring_slots=70000)
    for name in ("mla_attend_tree", "mla_attend_weight"):
        assert call(L, name, tall, n=65536) == UNS, name


def test_scales_and_workspaces(L):
    for bad in (0.0, -1.0, float("nan")):
        assert call(L, "mla_attend_tree", scale=bad) == ARG
        assert call(L, "mla_attend_weight", scale=bad) == ARG
    assert call(L, "mla_attend_tree", ws=None, ws_bytes=1 << 20) == ARG
    s = shape()
    need = L.mla_attend_tree_workspace_size(ctypes.byref(s), 4)
    if need:
        assert call(L, "mla_attend_tree", ws=FAKE, ws_bytes=need - 1) == ARG
    need = L.mla_cache_evict_workspace_size(ctypes.byref(s))
    # a count per sequence, and two lists of half the ring
    assert need == 4 * (64 + 64 * 2 * (8192 // 2 + 1))
    for name in ("mla_tree_accept", "mla_cache_evict"):
        assert call(L, name, ws_bytes=need - 1) == ARG
    assert L.mla_cache_evict_workspace_size(ctypes.byref(shape(batch=0))) == 0


def test_evict_long_rings(L):
    long = shape(batch=1, ring_slots=(1 << 30) + 1)
    for name in ("mla_tree_accept", "mla_cache_evict"):
        assert call(L, name, long, ws_bytes=1 << 62) == UNS


def test_evict_budgets(L):
    for k in ("keep", "sink", "recent"):
        assert call(L, "mla_cache_evict", **{k: -1}) == ARG
    assert call(L, "mla_cache_evict", keep=8193) == RANGE


def test_binding_refuses_tensors_it_cannot_pass(monkeypatch):
    """The library sees pointers: host tensors, strided ones, other element sizes and other devices
    stop in the binding."""
    import torch

    import latent_kv_cache_write_b200 as mla

    class Fake:
        dtype, shape, device = torch.bfloat16, (4, 4), "cuda:1"

        def __init__(self, item=2, contiguous=True, dev=0):
            self.item, self.contiguous, self.dev = item, contiguous, dev

        def element_size(self):
            return self.item

        def is_contiguous(self):
            return self.contiguous

        def stride(self):
            return (4, 1)

        def get_device(self):
            return self.dev

        def data_ptr(self):
            return FAKE

    monkeypatch.setattr(mla, "_current_device", lambda: 0)
    assert [mla._arg(t, 2, 0) for t in (Fake(), None, 7)] == [FAKE, None, 7]
    for bad in (Fake(item=4), Fake(contiguous=False), Fake(dev=1), torch.zeros(4, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            mla._arg(bad, 2, 0)
    assert mla._arg(Fake(item=1), 0, 0) == FAKE
    for bad in (Fake(contiguous=False), Fake(dev=1), torch.zeros(4)):
        with pytest.raises(ValueError):
            mla._arg(bad, 0, 0)
    s = shape()
    with pytest.raises(ValueError):
        mla.mla_attend_tree(s, torch.zeros(4), 1, FAKE, FAKE, None, 0.1, FAKE, stream=0)
    with pytest.raises(ValueError):
        mla.mla_cache_evict(s, FAKE, 1, 0, 0, torch.zeros(3, dtype=torch.int32), FAKE, FAKE, FAKE, 1,
                            stream=0)
    host = torch.zeros(1 << 16, dtype=torch.uint8)              # a workspace of the host
    for call in (lambda: mla.mla_attend_tree(s, FAKE, 1, FAKE, FAKE, None, 0.1, FAKE, None, host,
                                             stream=0),
                 lambda: mla.mla_tree_accept(s, FAKE, 1, FAKE, FAKE, None, None, host, stream=0),
                 lambda: mla.mla_cache_evict(s, FAKE, 1, 0, 0, FAKE, FAKE, FAKE, host, stream=0)):
        with pytest.raises(ValueError):
            call()

"""Draft-tree calls at the edges of their arguments (no GPU: refused, or nothing to do)."""

import math

import pytest
import torch

import latent_kv_cache_write_b200 as mla
from latent_kv_cache_write_b200 import native
from tests.test_tree_abi import ARG, CALLS, FAKE, OK, L, call, shape  # noqa: F401

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


class Fake:
    """A contiguous tensor of the current device that no call may reach the library with."""

    def __init__(self, dtype, *size):
        self.dtype, self.size, self.shape, self.device = dtype, size, size, "cuda:0"

    def element_size(self):
        return self.dtype.itemsize

    def numel(self):
        return math.prod(self.size)

    def is_contiguous(self):
        return True

    def stride(self):
        return self.size

    def get_device(self):
        return 0

    def data_ptr(self):
        return FAKE


BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
N, D_MODEL = 4, 256


def tensors(s, name):
    """The call's tensors by name, of the dtypes and sizes it needs."""
    B, H, S, dc, dr, dn = s.batch, s.n_heads, s.ring_slots, s.d_latent, s.d_rope, s.d_nope
    el = BF if s.dtype == native.MLA_BF16 else F32
    need = dict(cache=(el, B, S, dc + dr), window=(I32, B, 3), token=(I32, B, N), position=(I32, B, S),
                h=(el, B, N, D_MODEL), w_dkv=(el, D_MODEL, dc), w_kr=(el, D_MODEL, dr),
                q_nope=(el, B, N, H, dn), q_rope=(el, B, N, H, dr), w_uk=(el, H, dn, dc),
                q_abs=(el, B, N, H, dc + dr), tree=(U8, B, N, N), o_lat=(el, B, N, H, dc),
                lse=(F32, B, N, H), query_weight=(F32, B, N), weight_in=(F32, B, S),
                weight_out=(F32, B, S), weight=(F32, B, S), accept=(U8, B, N),
                ws=(U8, 1 << 24))
    return {k: Fake(*need[k]) for k in CALLS[name] if k in need}


def bind(name, s, t):
    """The binding's call with these tensors."""
    numbers = dict(d_model=D_MODEL, n=N, scale=0.07, keep=4, sink=0, recent=0)
    args = [t.get(k, numbers.get(k)) for k in CALLS[name] if k != "ws_bytes"]
    getattr(mla, name)(s, *args, stream=0)


@pytest.fixture
def reached(monkeypatch):
    """Stands in for the library: the names of the calls that would have run."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or OK

    monkeypatch.setattr(mla, "_current_device", lambda: 0)
    monkeypatch.setattr(native, "lib", lambda: Library())
    return calls


@pytest.mark.parametrize("dtype", [native.MLA_BF16, native.MLA_F32])
@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_other_dtypes(reached, name, dtype):
    """Elements of the right size but of another type are no window, weight or cache."""
    s = shape(dtype=dtype, ring_slots=300, batch=2)
    bind(name, s, tensors(s, name))
    assert reached == [name]
    other = {BF: (torch.float16, torch.int16, F32), F32: (I32, BF), I32: (F32, torch.uint32, torch.int64),
             U8: (I32, torch.int16)}
    for k, v in tensors(s, name).items():
        for wrong in other[v.dtype] if k != "ws" else ():
            t = dict(tensors(s, name), **{k: Fake(wrong, *v.size)})
            with pytest.raises(ValueError, match="needed"):
                bind(name, s, t)
        if v.dtype == U8:
            bind(name, s, dict(tensors(s, name), **{k: Fake(torch.bool, *v.size)}))
    assert set(reached) == {name}


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_short_tensors(reached, name):
    """One element less than the call reads or writes; longer ones (a batch's largest) pass."""
    s = shape(ring_slots=300, batch=2)
    for k, v in tensors(s, name).items():
        if k == "ws":
            continue
        with pytest.raises(ValueError, match="needed"):
            bind(name, s, dict(tensors(s, name), **{k: Fake(v.dtype, math.prod(v.size) - 1)}))
        bind(name, s, dict(tensors(s, name), **{k: Fake(v.dtype, math.prod(v.size) + 7)}))
    assert set(reached) == {name}


@pytest.mark.parametrize("name", [n for n in CALLS if "ws" in CALLS[n]])
def test_binding_workspaces(reached, name):
    """A raw pointer needs a size, and a size has to lie inside the tensor."""
    s = shape(ring_slots=300, batch=2)
    args = {k: v for k, v in tensors(s, name).items() if k != "ws"}
    numbers = dict(n=N, scale=0.07, keep=4, sink=0, recent=0)
    head = [args.get(k, numbers.get(k)) for k in CALLS[name] if k not in ("ws", "ws_bytes")]
    run = lambda ws, size=None: getattr(mla, name)(s, *head, ws, size, stream=0)  # noqa: E731
    with pytest.raises(ValueError, match="needs workspace_bytes"):
        run(FAKE)
    with pytest.raises(ValueError, match="has 64 bytes"):
        run(Fake(U8, 64), 65)
    for ws in (FAKE, Fake(U8, 64), None):
        with pytest.raises(ValueError):
            run(ws, -1)                                 # (no size_t)
    assert not reached
    run(FAKE, 64)
    run(Fake(U8, 64), 63)
    run(Fake(F32, 16))
    run(None)
    assert reached == [name] * 4

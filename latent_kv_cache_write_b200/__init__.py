"""Absorbed multi-head latent attention over a sliding-window latent KV ring on B200.

Python face of ``libmla.so``: the calls of the C ABI under the same names, taking
``torch`` CUDA tensors (or raw device pointers) and enqueuing on the current CUDA
stream unless a stream is given.  PyTorch supplies device memory and streams only;
all arithmetic runs in the library's kernels.

One chunk step (bf16; B sequences, T new tokens of one frame written at token g0, the
chunk's queries attending to the n_keys window tokens starting at k0)::

    import latent_kv_cache_write_b200 as mla
    shape = mla.MlaShape(batch=B, n_heads=H, d_nope=128, d_latent=512, d_rope=64,
                         rope_pairs=(8, 12, 12), rope_theta=1e4, grid_h=gh, grid_w=gw,
                         ring_slots=S, dtype=mla.native.MLA_BF16)
    mla.mla_cache_write(shape, h, d_model, T, g0, w_dkv, w_kr, cache)   # ring [B, S, 576]
    mla.mla_absorb_q(shape, q_nope, q_rope, T, g0, w_uk, q_abs)          # [B, T, H, 576]
    ws = torch.empty(mla.mla_attend_workspace_size(shape, T, n_keys), dtype=torch.uint8,
                     device="cuda")
    mla.mla_attend(shape, q_abs, T, g0, cache, k0, n_keys, scale, o_lat, lse, ws)
    mla.mla_up_v(shape, o_lat, T, w_uv, out)                             # [B, T, H, 128]

A serving loop with draft trees and sequences of their own lengths keeps those on the device
(``window`` int32 [B, 3]: first slot, context rows, nodes) and runs, per step::

    mla.mla_tree_write(shape, h, d_model, n, window, token, w_dkv, w_kr, cache, position)
    mla.mla_tree_absorb_q(shape, q_nope, q_rope, n, token, w_uk, q_abs)
    mla.mla_attend_tree(shape, q_abs, n, cache, window, tree, scale, o_lat, lse, ws)
    mla.mla_up_v(shape, o_lat, n, w_uv, out)
    # ... choose the accepted nodes ...
    mla.mla_attend_weight(shape, q_abs, n, cache, window, tree, scale, lse, accepted.float(),
                          weight, weight)
    mla.mla_tree_accept(shape, cache, n, accepted, window, weight, position, ews)
    mla.mla_cache_evict(shape, cache, n_keep, n_sink, n_recent, window, weight, position, ews)

``mla_attend_materialised`` replaces the last three calls of the chunk step with the non-absorbed form;
``mla_cache_shift_frames`` re-indexes the window's RoPE keys by whole frames;
``mla_cache_quantise`` / ``mla_cache_dequantise`` convert ring rows to and from the
low-bit ring.  Errors raise ``MlaError`` with the library's status.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

from . import native
from .native import MLA_FIXED_SCRATCH_BYTES, MlaError, MlaShape, make_shape  # noqa: F401

__all__ = ["mla_cache_write", "mla_absorb_q", "mla_attend", "mla_attend_workspace_size",
           "mla_attend_fixed_scratch", "mla_attend_materialised", "mla_attend_quantised",
           "mla_cache_shift_frames",
           "mla_cache_quantise", "mla_cache_dequantise",
           "mla_tree_write", "mla_tree_absorb_q", "mla_attend_tree",
           "mla_attend_tree_workspace_size", "mla_attend_weight", "mla_tree_accept",
           "mla_cache_evict", "mla_cache_evict_workspace_size",
           "mla_attend_materialised_workspace_size", "mla_up_v", "mla_device_error",
           "mla_kernel_launches", "mla_device_error_info", "mla_check_wait_timeout", "make_shape",
           "MlaShape", "MlaError", "MLA_FIXED_SCRATCH_BYTES"]


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, current: Optional[int] = None) -> Optional[int]:
    if stream is None:
        # the handle alone: building a Stream object takes longer than a launch
        return _cuda()._cuda_getCurrentRawStream(_current_device() if current is None else current)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def mla_cache_write(shape: MlaShape, h, d_model: int, n_tok: int, first_tok: int, w_dkv, w_kr,
                    cache, slots_out=None, stream=None) -> None:
    native.check("mla_cache_write", native.lib().mla_cache_write(
        ctypes.byref(shape), _ptr(h), d_model, n_tok, first_tok, _ptr(w_dkv), _ptr(w_kr),
        _ptr(cache), _ptr(slots_out), _stream(stream)))


def mla_absorb_q(shape: MlaShape, q_nope, q_rope, n_q: int, q_first_tok: int, w_uk, q_abs,
                 stream=None) -> None:
    native.check("mla_absorb_q", native.lib().mla_absorb_q(
        ctypes.byref(shape), _ptr(q_nope), _ptr(q_rope), n_q, q_first_tok, _ptr(w_uk),
        _ptr(q_abs), _stream(stream)))


def mla_attend_workspace_size(shape: MlaShape, n_q: int, n_keys: int) -> int:
    return int(native.lib().mla_attend_workspace_size(ctypes.byref(shape), n_q, n_keys))


def mla_attend(shape: MlaShape, q_abs, n_q: int, q_first_tok: int, cache, k_first_tok: int,
               n_keys: int, softmax_scale: float, o_lat, lse=None, workspace=None,
               workspace_bytes: Optional[int] = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else (
            workspace.numel() * workspace.element_size())
    native.check("mla_attend", native.lib().mla_attend(
        ctypes.byref(shape), _ptr(q_abs), n_q, q_first_tok, _ptr(cache), k_first_tok, n_keys,
        softmax_scale, _ptr(o_lat), _ptr(lse), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def mla_attend_fixed_scratch(shape: MlaShape, q_abs, n_q: int, q_first_tok: int, cache,
                             k_first_tok: int, n_keys: int, softmax_scale: float, o_lat,
                             lse=None, stream=None) -> None:
    native.check("mla_attend_fixed_scratch", native.lib().mla_attend_fixed_scratch(
        ctypes.byref(shape), _ptr(q_abs), n_q, q_first_tok, _ptr(cache), k_first_tok, n_keys,
        softmax_scale, _ptr(o_lat), _ptr(lse), _stream(stream)))


def mla_cache_shift_frames(shape: MlaShape, cache, first_tok: int, n_tok: int,
                           delta_frames: int, stream=None) -> None:
    native.check("mla_cache_shift_frames", native.lib().mla_cache_shift_frames(
        ctypes.byref(shape), _ptr(cache), first_tok, n_tok, delta_frames, _stream(stream)))


def mla_cache_quantise(shape: MlaShape, cache, first_tok: int, n_tok: int, content_bits: int,
                       rope_bits: int, q_content, q_rope, scale_c, scale_r,
                       stream=None) -> None:
    native.check("mla_cache_quantise", native.lib().mla_cache_quantise(
        ctypes.byref(shape), _ptr(cache), first_tok, n_tok, content_bits, rope_bits,
        _ptr(q_content), _ptr(q_rope), _ptr(scale_c), _ptr(scale_r), _stream(stream)))


def mla_cache_dequantise(shape: MlaShape, q_content, q_rope, scale_c, scale_r,
                         content_bits: int, rope_bits: int, first_tok: int, n_tok: int, cache,
                         stream=None) -> None:
    native.check("mla_cache_dequantise", native.lib().mla_cache_dequantise(
        ctypes.byref(shape), _ptr(q_content), _ptr(q_rope), _ptr(scale_c), _ptr(scale_r),
        content_bits, rope_bits, first_tok, n_tok, _ptr(cache), _stream(stream)))


def mla_attend_quantised(shape: MlaShape, q_abs, n_q: int, q_first_tok: int, q_content, q_rope,
                         scale_c, scale_r, content_bits: int, rope_bits: int, k_first_tok: int,
                         n_keys: int, softmax_scale: float, o_lat, lse=None, workspace=None,
                         workspace_bytes: Optional[int] = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else (
            workspace.numel() * workspace.element_size())
    native.check("mla_attend_quantised", native.lib().mla_attend_quantised(
        ctypes.byref(shape), _ptr(q_abs), n_q, q_first_tok, _ptr(q_content), _ptr(q_rope),
        _ptr(scale_c), _ptr(scale_r), content_bits, rope_bits, k_first_tok, n_keys,
        softmax_scale, _ptr(o_lat), _ptr(lse), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def mla_attend_materialised_workspace_size(shape: MlaShape) -> int:
    return int(native.lib().mla_attend_materialised_workspace_size(ctypes.byref(shape)))


def mla_attend_materialised(shape: MlaShape, q_nope, q_rope, n_q: int, q_first_tok: int,
                            cache, k_first_tok: int, n_keys: int, softmax_scale: float, w_uk,
                            w_uv, out, lse=None, workspace=None,
                            workspace_bytes: Optional[int] = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else (
            workspace.numel() * workspace.element_size())
    native.check("mla_attend_materialised", native.lib().mla_attend_materialised(
        ctypes.byref(shape), _ptr(q_nope), _ptr(q_rope), n_q, q_first_tok, _ptr(cache),
        k_first_tok, n_keys, softmax_scale, _ptr(w_uk), _ptr(w_uv), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def mla_up_v(shape: MlaShape, o_lat, n_q: int, w_uv, out, stream=None) -> None:
    native.check("mla_up_v", native.lib().mla_up_v(
        ctypes.byref(shape), _ptr(o_lat), n_q, _ptr(w_uv), _ptr(out), _stream(stream)))


def _arg(t, elem, current: int, count: int = 0) -> Optional[int]:
    """Device pointer of a tensor of at least ``count`` elements that are ``elem``: a dtype, or any of
    so many bytes (0: of any size, for a workspace).  A tensor of the host or of another device than
    ``current``, the current one, one with strides of its own, one that is too short, and one of
    other elements raise ValueError: the library sees pointers only."""
    if t is None or type(t) is int:
        return t
    if ((t.dtype is elem or elem == 0 or elem == t.element_size()) and t.get_device() == current
            and t.is_contiguous() and (not count or t.numel() >= count)):
        return t.data_ptr()
    what = f"{elem or 'any'}-byte elements" if isinstance(elem, int) else f"{elem} elements"
    raise ValueError(f"a contiguous tensor with {what} ({count} at least) on cuda:{current}, the "
                     f"current device, is needed, not {t.dtype} {tuple(t.shape)} with strides "
                     f"{t.stride()} on {t.device}")


def _current_device() -> int:
    # (short calls are bound by what the host does for each: no more than it has to)
    return _cuda()._cuda_getDevice()


@functools.lru_cache(None)
def _cuda():
    import torch
    torch.cuda.init()
    return torch._C


@functools.lru_cache(None)
def _kinds(dtype: int):
    """The dtypes of a shape's storage tensors, of the integer and of the float32 arrays."""
    import torch
    return (torch.bfloat16 if dtype == native.MLA_BF16 else torch.float32, torch.int32,
            torch.float32)


def _work(workspace, workspace_bytes: Optional[int], current: int):
    """Pointer and size of a workspace: all of a tensor unless a size is given, which then has to be
    inside it; a raw pointer needs a size."""
    if workspace is None or type(workspace) is int:
        if workspace_bytes is None and workspace is not None:
            raise ValueError("a workspace given as a pointer needs workspace_bytes")
        size = workspace_bytes = workspace_bytes or 0
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace_bytes is None:
            workspace_bytes = size
    if not 0 <= workspace_bytes <= size:
        raise ValueError(f"workspace_bytes is {workspace_bytes}, the workspace has {size} bytes")
    return _arg(workspace, 0, current), workspace_bytes


def _ring(shape: MlaShape):
    """Elements of a [B, S] array and of the cache."""
    slots = shape.batch * shape.ring_slots
    return slots, slots * (shape.d_latent + shape.d_rope)


def mla_tree_write(shape: MlaShape, h, d_model: int, n_nodes: int, window, token, w_dkv, w_kr,
                   cache, position=None, stream=None) -> None:
    dev, (el, i32, f32), (slots, ring) = _current_device(), _kinds(shape.dtype), _ring(shape)
    B = shape.batch
    native.check("mla_tree_write", native.lib().mla_tree_write(
        ctypes.byref(shape), _arg(h, el, dev, B * n_nodes * d_model), d_model, n_nodes,
        _arg(window, i32, dev, 3 * B), _arg(token, i32, dev, B * n_nodes),
        _arg(w_dkv, el, dev, d_model * shape.d_latent), _arg(w_kr, el, dev, d_model * shape.d_rope),
        _arg(cache, el, dev, ring), _arg(position, i32, dev, slots), _stream(stream, dev)))


def mla_tree_absorb_q(shape: MlaShape, q_nope, q_rope, n_nodes: int, token, w_uk, q_abs,
                      stream=None) -> None:
    dev, (el, i32, f32) = _current_device(), _kinds(shape.dtype)
    rows, dn, dc, dr = (shape.batch * n_nodes * shape.n_heads, shape.d_nope, shape.d_latent,
                        shape.d_rope)
    native.check("mla_tree_absorb_q", native.lib().mla_tree_absorb_q(
        ctypes.byref(shape), _arg(q_nope, el, dev, rows * dn), _arg(q_rope, el, dev, rows * dr),
        n_nodes, _arg(token, i32, dev, shape.batch * n_nodes),
        _arg(w_uk, el, dev, shape.n_heads * dn * dc), _arg(q_abs, el, dev, rows * (dc + dr)),
        _stream(stream, dev)))


def mla_attend_tree_workspace_size(shape: MlaShape, n_nodes: int) -> int:
    return int(native.lib().mla_attend_tree_workspace_size(ctypes.byref(shape), n_nodes))


def mla_attend_tree(shape: MlaShape, q_abs, n_nodes: int, cache, window, tree,
                    softmax_scale: float, o_lat, lse=None, workspace=None,
                    workspace_bytes: Optional[int] = None, stream=None) -> None:
    dev, (el, i32, f32), (slots, ring) = _current_device(), _kinds(shape.dtype), _ring(shape)
    B, rows, dc = shape.batch, shape.batch * n_nodes * shape.n_heads, shape.d_latent
    native.check("mla_attend_tree", native.lib().mla_attend_tree(
        ctypes.byref(shape), _arg(q_abs, el, dev, rows * (dc + shape.d_rope)), n_nodes,
        _arg(cache, el, dev, ring), _arg(window, i32, dev, 3 * B),
        _arg(tree, 1, dev, B * n_nodes * n_nodes), softmax_scale, _arg(o_lat, el, dev, rows * dc),
        _arg(lse, f32, dev, rows), *_work(workspace, workspace_bytes, dev), _stream(stream, dev)))


def mla_attend_weight(shape: MlaShape, q_abs, n_nodes: int, cache, window, tree,
                      softmax_scale: float, lse, query_weight, weight_in, weight_out,
                      stream=None) -> None:
    dev, (el, i32, f32), (slots, ring) = _current_device(), _kinds(shape.dtype), _ring(shape)
    B, rows = shape.batch, shape.batch * n_nodes * shape.n_heads
    native.check("mla_attend_weight", native.lib().mla_attend_weight(
        ctypes.byref(shape), _arg(q_abs, el, dev, rows * (shape.d_latent + shape.d_rope)), n_nodes,
        _arg(cache, el, dev, ring), _arg(window, i32, dev, 3 * B),
        _arg(tree, 1, dev, B * n_nodes * n_nodes), softmax_scale, _arg(lse, f32, dev, rows),
        _arg(query_weight, f32, dev, B * n_nodes), _arg(weight_in, f32, dev, slots),
        _arg(weight_out, f32, dev, slots), _stream(stream, dev)))


def mla_cache_evict_workspace_size(shape: MlaShape) -> int:
    return int(native.lib().mla_cache_evict_workspace_size(ctypes.byref(shape)))


def mla_tree_accept(shape: MlaShape, cache, n_nodes: int, accept, window, weight, position,
                    workspace, workspace_bytes: Optional[int] = None, stream=None) -> None:
    dev, (el, i32, f32), (slots, ring) = _current_device(), _kinds(shape.dtype), _ring(shape)
    B = shape.batch
    native.check("mla_tree_accept", native.lib().mla_tree_accept(
        ctypes.byref(shape), _arg(cache, el, dev, ring), n_nodes,
        _arg(accept, 1, dev, B * n_nodes), _arg(window, i32, dev, 3 * B),
        _arg(weight, f32, dev, slots), _arg(position, i32, dev, slots),
        *_work(workspace, workspace_bytes, dev), _stream(stream, dev)))


def mla_cache_evict(shape: MlaShape, cache, n_keep: int, n_sink: int, n_recent: int, window,
                    weight, position, workspace, workspace_bytes: Optional[int] = None,
                    stream=None) -> None:
    dev, (el, i32, f32), (slots, ring) = _current_device(), _kinds(shape.dtype), _ring(shape)
    native.check("mla_cache_evict", native.lib().mla_cache_evict(
        ctypes.byref(shape), _arg(cache, el, dev, ring), n_keep, n_sink, n_recent,
        _arg(window, i32, dev, 3 * shape.batch), _arg(weight, f32, dev, slots),
        _arg(position, i32, dev, slots),
        *_work(workspace, workspace_bytes, dev), _stream(stream, dev)))


def mla_kernel_launches() -> int:
    """Kernels launched by the library so far in this process."""
    return int(native.lib().mla_kernel_launches())


def mla_device_error_info() -> list:
    """[status bits, wait site id, CTA index, (thread << 16 | block)] of the last
    device-side error reported by mla_device_error."""
    buf = (ctypes.c_uint32 * 4)()
    native.lib().mla_device_error_info(buf)
    return list(buf)


def mla_check_wait_timeout(stream=None) -> None:
    """Enqueue the diagnostic whose bounded wait must expire; mla_device_error on the same
    stream then reports MLA_ERR_TIMEOUT."""
    native.check("mla_check_wait_timeout", native.lib().mla_check_wait_timeout(_stream(stream)))


def mla_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device-side error status."""
    return int(native.lib().mla_device_error(_stream(stream)))

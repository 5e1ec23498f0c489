"""The calls of the compiled module ``_binding`` (csrc/binding.cpp) in Python, argument by argument:
for machines where it was not built, or not against the installed PyTorch.  The checks and refusals
are the same; a call takes 15 to 27 us on the host in place of 4 to 10.
"""
from __future__ import annotations

import math
import operator

import torch

from . import (_DT, BF16, E4M3, F32, _addr, _exponents, _gpu, _launch, _same, _workspace,
               decode_tree_workspace)

_MOST = (1 << 31) - 1
_PAGE_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}


def _whole(x, name: str) -> int:
    x = operator.index(x)
    if not -_MOST - 1 <= x <= _MOST:
        raise ValueError(f"{name} does not fit 32 bits: {x}")
    return x


def _tokens(t, name: str, lead, index: int, dtype):
    """Check q, k or v of a call, lead + [heads, d] on device `index` with packed heads and one
    distance between tokens (a view of a fused projection is fine); returns (heads, d, that
    distance in elements)."""
    if _gpu(t, name) != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(lead) + 2 or list(t.shape[:-2]) != lead:
        raise ValueError(f"{name} must be {lead} + [heads, d], got {list(t.shape)}")
    *rows, heads, d = t.shape
    if max(heads, d) > _MOST:
        raise ValueError(f"{name} is too large")
    if t.is_contiguous():
        return heads, d, heads * d
    *strides, head_step, last = t.stride()
    if last != 1 or (heads > 1 and head_step != d):
        raise ValueError(f"{name}: heads and their elements must be contiguous")
    step, count = heads * d, 1
    for size, stride in zip(reversed(rows), reversed(strides)):
        if size > 1:   # dimensions of size 1 may have any stride
            if count == 1:
                step = stride
            elif stride != count * step:
                raise ValueError(f"{name}: tokens must be evenly spaced")
            count *= size
    return heads, d, step


def _frequencies(inv_freq, index: int) -> int:
    """How many there are."""
    n = _same(inv_freq, "inv_freq", index, torch.float64).numel()
    if n > _MOST // 2:
        raise ValueError("inv_freq is too large")   # any other wrong size is the library's to refuse
    return n


def _check_axes(axes, half: int):
    if axes is not None and len(axes) != half:
        raise ValueError(f"axes must hold {half} values, one for each frequency, got {len(axes)}")


def rope(backward, q, k, inv_freq, positions, interleaved, factor, q_out, k_out, axes):
    some = k if q is None else q
    index = _gpu(some, "q and k")
    if some.dim() != 4:
        raise ValueError(f"q and k must be [B, N, heads, d], got {list(some.shape)}")
    B, N, _, d = some.shape
    if max(B, N) > _MOST:
        raise ValueError("too many tokens")
    lead, dtype = [B, N], some.dtype
    kind = _DT[dtype]
    results, pointers, sizes = [], [], []
    for name, t, o in (("q", q, q_out), ("k", k, k_out)):
        if t is None:
            if o is not None:
                raise ValueError(f"out for {name}, which is None")
            results.append(None)
            pointers.append((None, None))
            sizes.append((0, 0, 0))
            continue
        heads, dt, step = _tokens(t, name, lead, index, dtype)
        if dt != d:
            raise ValueError("q and k must have one head size")
        if o is None:
            o, out_step = torch.empty(t.shape, dtype=dtype, device=t.device), heads * d
        else:
            oh, od, out_step = _tokens(o, f"out for {name}", lead, index, dtype)
            if oh != heads or od != d:
                raise ValueError(f"out for {name} must be {list(t.shape)}, got {list(o.shape)}")
        results.append(o)
        # a tensor without elements (no tokens, no heads) has nothing to rotate; the other may
        pointers.append((t.data_ptr(), o.data_ptr()) if t.numel() else (None, None))
        sizes.append((heads, step, out_step))
    half = _frequencies(inv_freq, index)
    _check_axes(axes, half)
    more = ()
    if axes is not None:
        if positions is None:
            raise ValueError("axes without positions")
        shape = _same(positions, "positions", index, torch.int32).shape
        if len(shape) != 3 or shape[1] != B or shape[2] != N or shape[0] > _MOST:
            raise ValueError(f"positions must be [axes, {B}, {N}], got {list(shape)}")
        more = (axes, shape[0])
    elif positions is not None and _same(positions, "positions", index, torch.int32).numel() != B * N:
        raise ValueError(f"positions must hold {B * N} values, got {positions.numel()}")
    interleaved, factor = bool(interleaved), float(factor)
    if pointers[0][0] or pointers[1][0]:
        where = "swiattn_rope" + ("" if axes is None else "_axes") + ("_backward" if backward else "")
        (Hq, qs, qos), (Hkv, ks, kos) = sizes
        _launch(where, index, pointers[0][0], pointers[1][0], _addr(positions), *more,
                inv_freq.data_ptr(), pointers[0][1], pointers[1][1], B, N, Hq, Hkv, d, 2 * half,
                interleaved, factor, qs, ks, qos, kos, kind)
    return results[0], results[1]


def _pools(k_pages, v_pages, k_exp, v_exp, index: int, layered: bool):
    """Check page pools of one layer [num_pages, page_size, Hkv, d] or, if `layered`, also of several
    [layers, num_pages, page_size, Hkv, d]; returns the pointers and (layers, num_pages, page_size,
    Hkv, d, page type)."""
    dtype = _same(k_pages, "k_pages", index).dtype
    shape = k_pages.shape
    if _same(v_pages, "v_pages", index, dtype).shape != shape or not (
            len(shape) == 4 or (layered and len(shape) == 5)):
        raise ValueError("k_pages and v_pages must both be " + (
            "[layers, num_pages, page_size, Hkv, d] or " if layered else "") + "[num_pages, page_size, Hkv, d]")
    if max(shape) > _MOST:
        raise ValueError("k_pages is too large")
    kind = _PAGE_TYPES.get(dtype)
    if kind is None:
        raise ValueError(f"pages must be float32, bfloat16 or float8_e4m3fn, got {dtype}")
    num_pages, page_size, Hkv, d = shape[-4:]
    ke = ve = None
    if kind == E4M3:
        want = (*shape[:-4], num_pages, Hkv, page_size)
        _exponents(k_exp, "k_exp", index, want)
        _exponents(v_exp, "v_exp", index, want)
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    return ((k_pages.data_ptr(), v_pages.data_ptr(), ke, ve),
            (shape[0] if len(shape) == 5 else 1, num_pages, page_size, Hkv, d, kind))


def _sequences(block_table, seq_lens, index: int):
    """Check block_table [B, max_pages] and seq_lens [B]; returns (B, max_pages)."""
    B = _same(seq_lens, "seq_lens", index, torch.int32).numel()
    table = _same(block_table, "block_table", index, torch.int32).shape
    if len(table) != 2 or table[0] != B or max(B, table[1]) > _MOST:
        raise ValueError(f"block_table must be [{B}, max_pages]")
    return B, table[1]


def _ints(t, name: str, index: int, count: int):
    if _same(t, name, index, torch.int32).numel() != count:
        raise ValueError(f"{name} must hold {count} values, got {t.numel()}")
    return t.data_ptr()


def append_paged(q, k, v, k_pages, v_pages, block_table, seq_lens, inv_freq, starts, interleaved,
                 factor, k_exp, v_exp, out, positions, axes):
    index = _gpu(k, "k")
    if k.dim() != 3:
        raise ValueError(f"k must be [T, Hkv, d], got {list(k.shape)}")
    T, dtype = k.shape[0], k.dtype
    kind, lead = _DT[dtype], [T]
    if T > _MOST:
        raise ValueError("too many tokens")
    Hkv, d, ks = _tokens(k, "k", lead, index, dtype)
    vh, vd, vs = _tokens(v, "v", lead, index, dtype)
    if vh != Hkv or vd != d:
        raise ValueError("k and v must have one shape")
    Hq, qs = 0, 0
    if q is not None:
        Hq, qd, qs = _tokens(q, "q", lead, index, dtype)
        if qd != d:
            raise ValueError("q and k must have one head size")
        if out is None:
            out = torch.empty(q.shape, dtype=dtype, device=q.device)
        elif _same(out, "out", index, dtype).shape != q.shape:
            raise ValueError(f"out must be {list(q.shape)}, got {list(out.shape)}")
    elif out is not None:
        raise ValueError("out without q")
    if _same(k_pages, "k_pages", index).dtype not in (dtype, torch.float8_e4m3fn):
        raise ValueError(f"pages must be {dtype} or float8_e4m3fn, got {k_pages.dtype}")
    pools, (_, num_pages, page_size, ph, pd, page_kind) = _pools(k_pages, v_pages, k_exp, v_exp, index, False)
    if ph != Hkv or pd != d:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]")
    B, max_pages = _sequences(block_table, seq_lens, index)
    at = None if starts is None else _ints(starts, "starts", index, B + 1)
    half = 0 if inv_freq is None else _frequencies(inv_freq, index)
    where, more = "swiattn_append_paged", ()
    if positions is not None or axes is not None:
        if inv_freq is None or positions is None:
            raise ValueError("positions turn by inv_freq, and axes are of positions")
        given = _same(positions, "positions", index, torch.int32).shape
        _check_axes(axes, half)
        if len(given) != (1 if axes is None else 2) or given[-1] != T or given[0] > _MOST:
            raise ValueError(f"positions must be [{T}], or [axes, {T}] with axes, got {list(given)}")
        where = "swiattn_append_paged_at"
        more = (positions.data_ptr(), axes, 1 if axes is None else given[0])
    _launch(where, index, _addr(q), k.data_ptr(), v.data_ptr(), at, seq_lens.data_ptr(),
            block_table.data_ptr(), *more, _addr(inv_freq), None if q is None else out.data_ptr(),
            *pools, T, B, max_pages, page_size, num_pages, Hq, Hkv, d, 2 * half, bool(interleaved),
            float(factor), qs, ks, vs, kind, page_kind)
    return out


def _parents(parents, index: int):
    """Check parents [T] or None; returns (pointer, T or None)."""
    if parents is None:
        return None, None
    if _same(parents, "parents", index, torch.int32).dim() != 1:
        raise ValueError("parents must be [T]")
    return parents.data_ptr(), parents.numel()


def decode_tree(q, k_pages, v_pages, block_table, seq_lens, starts, parents, gate, W, scale, out,
                want_lse, workspace, n_anchor, k_exp, v_exp):
    index = _gpu(q, "q")
    _same(q, "q", index)
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, d], got {list(q.shape)}")
    T, Hq, d = q.shape
    kind = _DT[q.dtype]
    if max(T, Hq, d) > _MOST:
        raise ValueError("q is too large")
    pools, (_, num_pages, page_size, Hkv, dk, page_kind) = _pools(k_pages, v_pages, k_exp, v_exp, index, False)
    if dk != d:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]")
    B, max_pages = _sequences(block_table, seq_lens, index)
    at = _ints(starts, "starts", index, B + 1)
    parent, count = _parents(parents, index)
    if count not in (None, T) or _same(gate, "gate", index, torch.uint8).numel() != T:
        raise ValueError(f"parents and gate must hold {T} values")
    W, n_anchor = _whole(W, "W"), _whole(n_anchor, "n_anchor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    elif _same(out, "out", index, q.dtype).shape != q.shape:
        raise ValueError(f"out must be {list(q.shape)}, got {list(out.shape)}")
    lse = torch.empty((T, Hq), device=q.device, dtype=torch.float32) if want_lse else None
    if workspace is None:
        workspace = _workspace(decode_tree_workspace(T, B, Hq, Hkv, d, kind), q.device, None)
    else:
        _same(workspace, "workspace", index, torch.uint8)
    _launch("swiattn_decode_tree", index, q.data_ptr(), *pools, block_table.data_ptr(),
            seq_lens.data_ptr(), at, parent, gate.data_ptr(), out.data_ptr(), _addr(lse), T, B,
            max_pages, page_size, num_pages, Hq, Hkv, d, W, n_anchor, scale, kind, page_kind,
            workspace.data_ptr(), workspace.numel())
    return (out, lse) if want_lse else out


def accept_tree(k_pages, v_pages, block_table, seq_lens, starts, parents, leaf, k_exp, v_exp, out):
    index = _gpu(k_pages, "k_pages")
    pools, (layers, num_pages, page_size, Hkv, d, kind) = _pools(k_pages, v_pages, k_exp, v_exp, index, True)
    B, max_pages = _sequences(block_table, seq_lens, index)
    at = _ints(starts, "starts", index, B + 1)
    parent, count = _parents(parents, index)
    T = _MOST if count is None else count
    if T > _MOST:
        raise ValueError("too many tokens")
    path = _ints(leaf, "leaf", index, B)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=k_pages.device)
    _launch("swiattn_accept_tree", index, *pools, block_table.data_ptr(), seq_lens.data_ptr(), at,
            parent, path, _ints(out, "out", index, B), layers, T, B, max_pages, page_size, num_pages,
            Hkv, d, kind)
    return out


def fork_paged(k_pages, v_pages, block_table, seq_lens, source, new_page, k_exp, v_exp, table, lens):
    index = _gpu(k_pages, "k_pages")
    pools, (layers, num_pages, page_size, Hkv, d, kind) = _pools(k_pages, v_pages, k_exp, v_exp, index, True)
    B, max_pages = _sequences(block_table, seq_lens, index)
    C = _same(source, "source", index, torch.int32).numel()
    if C > _MOST:
        raise ValueError("too many children")
    own = _ints(new_page, "new_page", index, C)
    if table is None and lens is None:
        table = torch.empty((C, max_pages), dtype=torch.int32, device=k_pages.device)
        lens = torch.empty(C, dtype=torch.int32, device=k_pages.device)
    elif _same(table, "out", index, torch.int32).shape != (C, max_pages):
        raise ValueError(f"out must be [{C}, {max_pages}] and [{C}]")
    _launch("swiattn_fork_paged", index, *pools, block_table.data_ptr(), seq_lens.data_ptr(),
            source.data_ptr(), own, table.data_ptr(), _ints(lens, "out", index, C), layers, B, C,
            max_pages, page_size, num_pages, Hkv, d, kind)
    return table, lens

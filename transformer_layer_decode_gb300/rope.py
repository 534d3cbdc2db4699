"""Rotary positions (the dec_rope_ calls of include/dec.h).

:class:`Rotary` is a model's rotation: which dimensions turn, in which pairs and
how fast.  It rotates the rows of many sequences here, and the keys and queries
of a step in :meth:`.kv.KVCache.append_rotated`.  Calls are queued on a stream
and wait for nothing.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import dec

DEC_ROPE_HALF, DEC_ROPE_PAIRS = 0, 1
DEC_ROPE_PLAIN, DEC_ROPE_LINEAR, DEC_ROPE_NTK, DEC_ROPE_YARN, DEC_ROPE_YARN_INDEX = 0, 1, 2, 3, 4

LAYOUTS = {"half": DEC_ROPE_HALF, "interleaved": DEC_ROPE_PAIRS}
SCALINGS = {None: DEC_ROPE_PLAIN, "linear": DEC_ROPE_LINEAR, "ntk": DEC_ROPE_NTK, "yarn": DEC_ROPE_YARN}
RAMPS = {"turns": DEC_ROPE_YARN, "index": DEC_ROPE_YARN_INDEX}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class RopeDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("steps", ctypes.c_void_p)]


class Rotary:
    """The rotation of the first `rot_dim` (all) dimensions of heads of `head_dim`.

    layout: "half" turns dimensions (i, i + rot_dim / 2), "interleaved" (2 i, 2 i + 1).  The frequencies, in
    radians per position, are theta^(-2 i / rot_dim), made slower for long contexts by `scaling`: "linear"
    divides them by `factor`; "ntk" enlarges theta so that the slowest is divided by it and the fastest
    stays; "yarn" keeps those that turn `fast` times or more over `context` positions, divides those that
    turn `slow` times or less, and multiplies the rotated values by 0.1 log(factor) + 1.  Between these two `ramp`
    says how: "turns", in proportion to a frequency's turns, which is the paper's formula, or "index", in
    proportion to its number, between whole ones.  Models that are published with this scaling were trained with
    "index": load them with ramp="index", since two dozen of 64 frequencies differ, some by a factor of two.
    Or the frequencies are given, `frequencies` [rot_dim / 2], and `magnitude`, which otherwise overrides the
    scaling's, with them.
    A captured graph needs the rotation alive, as it does a cache.
    """

    def __init__(self, head_dim: int, *, rot_dim: int | None = None, layout: str = "half", theta: float = 1e4,
                 scaling: str | None = None, factor: float = 1.0, context: float = 0.0, slow: float = 1.0,
                 fast: float = 32.0, ramp: str = "turns", frequencies=None, magnitude: float | None = None, device=None,
                 lib_path: str | None = None):
        if layout not in LAYOUTS:
            raise ValueError(f"layout {layout!r}: one of {sorted(LAYOUTS)}")
        if scaling not in SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {[k for k in SCALINGS if k]} or None")
        if ramp not in RAMPS or (ramp != "turns" and scaling != "yarn"):
            raise ValueError(f"ramp {ramp!r}: one of {sorted(RAMPS)}, of scaling 'yarn'")
        rot_dim = head_dim if rot_dim is None else rot_dim
        if not (8 <= head_dim <= 1024 and head_dim % 8 == 0):
            raise ValueError(f"head_dim {head_dim}: a multiple of 8, 8..1024")
        if not (2 <= rot_dim <= head_dim and rot_dim % 2 == 0):
            raise ValueError(f"rot_dim {rot_dim}: even, 2..{head_dim}")
        self.lib = dec.load_library(lib_path or dec.LIB_PATH)
        if frequencies is None:
            self.frequencies, m = np.empty(rot_dim // 2), ctypes.c_float()
            kind = RAMPS[ramp] if scaling == "yarn" else SCALINGS[scaling]
            self._check(self.lib.dec_rope_frequencies(rot_dim, theta, kind, factor, context, slow, fast,
                                                      self.frequencies.ctypes.data, ctypes.byref(m)))
            magnitude = m.value if magnitude is None else magnitude
        else:
            if scaling is not None:
                raise ValueError("frequencies that are given are not scaled")
            self.frequencies = np.array(frequencies, np.float64)
            if self.frequencies.shape != (rot_dim // 2,):
                raise ValueError(f"frequencies: {rot_dim // 2} of them are wanted")
            magnitude = 1.0 if magnitude is None else magnitude
        if not abs(magnitude) < 3.4e38:
            raise ValueError(f"magnitude {magnitude}: a finite fp32 number is wanted")
        steps = np.empty(rot_dim // 2, np.uint64)
        self._check(self.lib.dec_rope_steps(self.frequencies.ctypes.data, rot_dim // 2, steps.ctypes.data))
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError("a rotation belongs to a CUDA device")
        self.head_dim, self.rot_dim, self.layout, self.magnitude = head_dim, rot_dim, layout, magnitude
        self.steps = torch.from_numpy(steps.view(np.int64)).to(device)  # (finished when this returns: pageable memory)
        self.device, self._index = self.steps.device, self.steps.device.index
        self.desc = RopeDesc(head_dim, rot_dim, LAYOUTS[layout], magnitude, self.steps.data_ptr())
        self._ref = ctypes.byref(self.desc)
        self._fast, self._context = dec.load_calls(), None
        if self._fast is not None:
            self._context = self._fast.context(ctypes.addressof(self.desc), self._index, 0, head_dim,
                                               dec.address_of(self.lib.dec_rope_rotate))

    def _check(self, rc: int):
        if rc != dec.DEC_OK:
            raise dec.DecError(rc, self.lib.dec_last_error(None).decode())

    def _rows(self, name, t):
        """(address, type, elements from row to row) of a [n, heads, head_dim] tensor with whole rows."""
        shape, d = t.shape, self.head_dim
        if len(shape) == 3 and shape[2] == d and shape[1] and t.device == self.device:
            step, type_ = t.stride(), _TYPES.get(t.dtype)
            if type_ is not None and step[2] == 1 and (step[1] == d or shape[1] == 1):
                return t.data_ptr(), type_, step[0] if shape[0] > 1 else shape[1] * d
        raise ValueError(f"{name}: a float32 or bfloat16 tensor [n, heads, {d}] on {self.device} with contiguous rows is "
                         "wanted")

    def rotate(self, x, positions=None, *, out=None, backward: bool = False, stream=None):
        """Row t of x ([n, heads, head_dim]) rotated by positions[t] (int32; without them, by t).  A row with a
        negative position is skipped, and keeps what `out` holds (zeros where that is made here).  `out` may be
        x.  backward: by the negative angles, the gradient of a rotation.  Autograd sees neither: the result of an x
        that requires a gradient has none, and an autograd function that wants one calls both."""
        if stream is None and out is not None and self._context is not None:  # (marshalled where plainly right, as KVCache's calls are)
            rc = self._fast.rotate(self._context, x, positions, out, bool(backward))
            if rc is not None:
                if rc:
                    self._check(rc)
                return out
        xp, xt, xs = self._rows("x", x)
        n, heads = x.shape[0], x.shape[1]
        if positions is not None and (positions.dtype != torch.int32 or positions.shape != (n,)
                                      or not positions.is_contiguous() or positions.device != self.device):
            raise ValueError(f"positions: {n} contiguous int32 numbers on {self.device} are wanted")
        handle = _raw_stream(self._index) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        if out is None:
            make = torch.empty if positions is None else torch.zeros
            if stream is None:
                out = make(x.shape, dtype=x.dtype, device=self.device)
            else:  # its memory, and what fills it, belong to that stream
                on = torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) else stream
                with torch.cuda.stream(on):
                    out = make(x.shape, dtype=x.dtype, device=self.device)
        op, ot, os_ = self._rows("out", out)
        if ot != xt or out.shape != x.shape:
            raise ValueError("out: the type and shape of x are wanted")
        args = (self._ref, xp, op, xt, xs, os_, None if positions is None else positions.data_ptr(), n, heads,
                int(backward), handle)
        if _current_device() == self._index:
            rc = self.lib.dec_rope_rotate(*args)
        else:
            with torch.cuda.device(self.device):
                rc = self.lib.dec_rope_rotate(*args)
        if rc:
            self._check(rc)
        return out

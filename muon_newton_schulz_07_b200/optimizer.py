"""PyTorch-facing wrapper of libmuon: torch allocates the workspace and provides the stream.

    step = MuonStep([(1536, 1536), (1536, 6144), ...], dtype=torch.bfloat16)
    step(W_list, G_list, M_list, lr=0.02, beta=0.95)      # W and M updated in place

Only argument checking and pointer marshalling happen here; the optimizer step
itself runs in libmuon's kernels on the current CUDA stream.
"""
from __future__ import annotations

import torch

from . import binding as B

QUINTIC = (3.4445, -4.7750, 2.0315)

_VIEW_TYPES = {torch.bfloat16: B.MUON_BF16, torch.float32: B.MUON_FP32, torch.float16: B.MUON_FP16}


def _entries(shapes):
    """(count, rows, cols, shape a tensor of the entry has) of (rows, cols) matrices and (count, rows, cols) stacks."""
    out = []
    for s in shapes:
        s = tuple(int(x) for x in s)
        if len(s) not in (2, 3):
            raise ValueError(f"a shape is (rows, cols) or (count, rows, cols): got {s}")
        out.append((s if len(s) == 3 else (1,) + s) + (s,))
    return out


def _views(tensors, entries, device, name, dtype=None, by_rows=False):
    """Views of tensors that may be strided; dtype None: any of bf16, fp16 and fp32."""
    if len(tensors) != len(entries):
        raise ValueError(f"{name}: expected {len(entries)} tensors, got {len(tensors)}")
    out = []
    for t, (count, rows, cols, shape) in zip(tensors, entries):
        dt = t.dtype
        if t.shape != shape or t.device != device or (dt is not dtype if dtype else dt not in _VIEW_TYPES):
            raise ValueError(f"{name}: tensor {tuple(t.shape)} {t.dtype} {t.device} does not match {shape} "
                             f"{dtype or 'bf16, fp16 or fp32'} {device}")
        st = t.stride()
        bs, rs, cs = st if len(st) == 3 else (0,) + st
        if cs != 1 and cols != 1 and (by_rows or not (rs == 1 or rows == 1)):
            raise ValueError(f"{name}: a tensor of strides {st} is not stored by rows"
                             + ("" if by_rows else " or by columns"))
        out.append(B.pack_view(t.data_ptr(), count, bs, rs, cs, _VIEW_TYPES[dt]))
    return b"".join(out)


def _device(device):
    dev = torch.device(device if device is not None else "cuda")
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


def _stream(device, stream):
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream(device).cuda_stream, without a Stream object (2 us of a call's 10 on the host)
    return torch._C._cuda_getCurrentRawStream(device.index)


class QuantizedState:
    """8-bit optimizer state: codes (int8 or e4m3), and one fp32 scale for each 128 columns of a row.

        state = QuantizedState([(768, 768), (12, 64, 768)], fmt="int8")    # zero
        state.write(tensors, seed=step)                                     # quantise
        state.read(tensors)                                                 # read back
        step(W, G, state, seed=t)                                           # a MuonStep's momentum (mode="half")

    Shapes are (rows, cols) matrices or (count, rows, cols) stacks.  `codes` and `scales` are lists of tensors
    of those shapes, to be saved, loaded and sharded by rows like any other.  Rounding is to nearest even, or, with
    a seed, stochastic: unbiased, from a generator of the seed and the value's place; give every call another seed.
    Int8 is finer where the values of a block are alike, e4m3 keeps small values beside large ones.
    """

    FORMATS = {"int8": (B.MUON_STATE_INT8, torch.int8), "e4m3": (B.MUON_STATE_E4M3, torch.float8_e4m3fn)}
    BLOCK = B.MUON_STATE_BLOCK

    def __init__(self, shapes, fmt: str = "int8", device=None):
        if fmt not in self.FORMATS:
            raise ValueError(f"fmt must be one of {sorted(self.FORMATS)}")
        self.fmt = fmt
        self._fmt, self._type = self.FORMATS[fmt]
        self._entries = _entries(shapes)
        self.shapes = [e[3] for e in self._entries]
        self._scale_shapes = [s[:-1] + (-(-s[-1] // self.BLOCK),) for s in self.shapes]
        self.device = dev = _device(device)
        self.codes = [torch.zeros(s, dtype=torch.uint8, device=dev).view(self._type) for s in self.shapes]
        self.scales = [torch.zeros(s, dtype=torch.float32, device=dev) for s in self._scale_shapes]

    def _states(self):
        out = []
        code, device = self._type, self.device
        for q, s, (count, rows, cols, shape), scales in zip(self.codes, self.scales, self._entries, self._scale_shapes,
                                                             strict=True):
            if q.shape != shape or q.dtype is not code or q.device != device or not q.is_contiguous():
                raise ValueError(f"codes: tensor {tuple(q.shape)} {q.dtype} {q.device} does not match {shape} {code} "
                                 f"{self.device} (contiguous)")
            if s.shape != scales or s.dtype is not torch.float32 or s.device != device or not s.is_contiguous():
                raise ValueError(f"scales: tensor {tuple(s.shape)} {s.dtype} {s.device} does not match {shape}, a scale "
                                 f"for {self.BLOCK} columns, torch.float32 {self.device} (contiguous)")
            out.append(B.pack_state(q.data_ptr(), s.data_ptr(), count, rows, cols))
        return b"".join(out)

    def _side(self, tensors, name):
        if len(tensors) > 1 and any(t.dtype is not tensors[0].dtype for t in tensors):
            raise ValueError(f"{name}: tensors of one call have one dtype")
        return _views(tensors, self._entries, self.device, name, by_rows=True)

    def write(self, X, seed=None, stream=None) -> None:
        """Quantise X (bf16, fp16 or fp32, stored by rows) into this state, on the current stream or `stream`."""
        self._call(B.muon_state_quantize, self._side(X, "X"), self._states(), len(self.shapes), self._fmt, seed,
                   _stream(self.device, stream))

    def read(self, out, stream=None) -> None:
        """Read this state back into the tensors of `out` (bf16, fp16 or fp32, stored by rows)."""
        self._call(B.muon_state_dequantize, self._states(), self._side(out, "out"), len(self.shapes), self._fmt,
                   _stream(self.device, stream))

    def _call(self, f, *args):
        if torch._C._cuda_getDevice() == self.device.index:
            f(*args)
        else:  # the library launches on the current device
            with torch.cuda.device(self.device):
                f(*args)


class MuonStep:
    """A Muon step for one fixed list of matrix shapes, bound to one CUDA device.

    A shape is (rows, cols), or (count, rows, cols) for a stack of equal matrices, each stepped by itself (experts,
    attention heads).  mode: "fast" (bf16 operands), "half" (fp16 operands: an eighth of the rounding error in about
    the same time; takes strided views, coefficients per iteration and 8-bit momentum) or "fp32_ref" (slow, exact).
    """

    SCHEDULES = {"auto": B.MUON_SCHEDULE_AUTO, "staged": B.MUON_SCHEDULE_STAGED, "fused": B.MUON_SCHEDULE_FUSED,
                 "split": B.MUON_SCHEDULE_SPLIT}

    def __init__(self, shapes, dtype=torch.bfloat16, mode: str = "fast", device=None, schedule: str = "auto"):
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dtype must be torch.bfloat16 or torch.float32")
        if mode not in ("fast", "half", "fp32_ref"):
            raise ValueError("mode must be 'fast', 'half' or 'fp32_ref'")
        self._entries = _entries(shapes)
        self.shapes = [e[3] for e in self._entries]
        matrices = [(rows, cols) for count, rows, cols, _ in self._entries for _ in range(count)]
        self.mode = mode
        self.dtype = dtype
        self.device = _device(device)
        self._dt = B.MUON_BF16 if dtype == torch.bfloat16 else B.MUON_FP32
        self._mode = {"fast": B.MUON_MODE_FAST, "half": B.MUON_MODE_HALF, "fp32_ref": B.MUON_MODE_FP32_REF}[mode]
        nbytes = B.muon_workspace_size(matrices, self._dt, self._mode)
        self._n = len(matrices)
        self.workspace_bytes = nbytes
        with torch.cuda.device(self.device):
            self._ws = torch.empty(nbytes + 1024, dtype=torch.uint8, device=self.device)
            base = self._ws.data_ptr()
            self._ws_ptr = (base + 1023) // 1024 * 1024
            # the block may be one that this stream's earlier work still uses; muon_create fills it on another stream
            torch.cuda.current_stream(self.device).synchronize()
            self.handle = B.muon_create(matrices, self._dt, self._mode, self._ws_ptr, nbytes)
        self._streams = {_stream(self.device, None)}
        self.n_groups, _ = B.muon_get_plan(self.handle, 5)
        if schedule != "auto":
            self.set_schedule(schedule)

    def _on(self, stream):
        """The stream of a call.  The workspace's block stays allocated until that stream's work on it is done."""
        raw = _stream(self.device, stream)
        if raw not in self._streams:
            self._streams.add(raw)
            self._ws.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
        return raw

    def set_schedule(self, schedule: str) -> None:
        """'auto', 'staged' (one launch per Newton-Schulz stage), 'fused' (every iteration in one launch)
        or 'split' (the fused kernel's tiles, one launch per stage)."""
        if schedule not in self.SCHEDULES:
            raise ValueError(f"schedule must be one of {sorted(self.SCHEDULES)}")
        B.muon_set_schedule(self.handle, self.SCHEDULES[schedule])

    def launches_per_step(self, ns_steps: int = 5) -> int:
        return B.muon_get_plan(self.handle, ns_steps)[1]

    def _check(self, tensors, name):
        if len(tensors) != len(self.shapes):
            raise ValueError(f"{name}: expected {len(self.shapes)} tensors, got {len(tensors)}")
        for t, s in zip(tensors, self.shapes):
            if tuple(t.shape) != s or t.dtype != self.dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{name}: tensor {tuple(t.shape)} {t.dtype} {t.device} does not match {s} "
                                 f"{self.dtype} {self.device} (contiguous)")
        # one pointer a matrix: a stack holds its matrices back to back
        return [t.data_ptr() + e * rows * cols * t.element_size()
                for t, (count, rows, cols, _) in zip(tensors, self._entries) for e in range(count)]

    def _coefficients(self, abc, ns_steps):
        """(abc for the hyper-parameters, iterations); a list of triples, one per iteration, goes to the handle."""
        # (a tensor of no dimensions has a len)
        scalars = (True,) * 3 if abc is QUINTIC else [not hasattr(t, "__len__") or getattr(t, "ndim", 1) == 0 for t in abc]
        if len(abc) == 3 and all(scalars):
            if self.mode == "half":
                B.muon_set_coefficients(self.handle, ())
            return abc, 5 if ns_steps is None else ns_steps
        if self.mode != "half":
            raise ValueError("abc must be one (a, b, c): coefficients per iteration need mode='half'")
        if any(one or len(t) != 3 for one, t in zip(scalars, abc)) or (ns_steps is not None and ns_steps != len(abc)):
            raise ValueError("abc must be one (a, b, c), or one for each of the ns_steps iterations")
        B.muon_set_coefficients(self.handle, abc)
        return QUINTIC, len(abc)

    def _momentum_state(self, state):
        if state.shapes != self.shapes or state.device != self.device:
            raise ValueError(f"state: shapes {state.shapes} on {state.device} do not match {self.shapes} on {self.device}")
        return state._states()

    def __call__(self, W, G, M, lr=0.02, beta=0.95, weight_decay=0.0, eps=1e-7, abc=QUINTIC, nesterov=True,
                 ns_steps=None, stream=None, seed=None):
        """One step: W and M updated in place.

        M is a list of tensors, or a QuantizedState (mode "half"; `seed` then makes its rounding stochastic, and
        W and G may be strided: G stored by rows, W by rows or by columns).  abc is one coefficient triple for
        ns_steps iterations (5 by default) or, in mode "half", a list with one for each iteration.
        """
        quantized = isinstance(M, QuantizedState)
        if seed is not None and not quantized:
            raise ValueError("seed is for a QuantizedState")
        if quantized and self.mode != "half":
            raise ValueError("a QuantizedState needs mode='half'")
        if quantized:
            states = self._momentum_state(M)
            w = _views(W, self._entries, self.device, "W", self.dtype)
            g = _views(G, self._entries, self.device, "G", self.dtype, by_rows=True)
            abc, ns_steps = self._coefficients(abc, ns_steps)
            hp = B.make_hparams(lr, beta, weight_decay, eps, abc, nesterov, ns_steps)
            B.muon_step_state(self.handle, w, g, states, len(self.shapes), M._fmt, hp, seed, self._on(stream))
            return
        abc, ns_steps = self._coefficients(abc, ns_steps)
        hp = B.make_hparams(lr, beta, weight_decay, eps, abc, nesterov, ns_steps)
        B.muon_step(self.handle, self._check(W, "W"), self._check(G, "G"), self._check(M, "M"), hp, self._on(stream))

    def step_from_host(self, W, G_host, M, stream=None, **hp):
        """A step whose gradients are in pinned host memory.

        The host-to-device copy of G runs on a side stream into one of two device buffers,
        so it overlaps the previous step's kernels; the step itself waits for its copy.  The
        buffer is reused two steps later, once the step that read it has finished.  Keyword
        arguments are those of __call__.
        """
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if getattr(self, "_gbuf", None) is None:
            self._gbuf = [[torch.empty(sh, dtype=self.dtype, device=self.device) for sh in self.shapes]
                          for _ in range(2)]
            self._copy_stream = torch.cuda.Stream(self.device)
            self._copy_stream.wait_stream(torch.cuda.current_stream(self.device))  # earlier work on these blocks
            self._buf_free = [None, None]
            self._buf_streams = {torch.cuda.current_stream(self.device).cuda_stream}
            self._nfed = 0
        if len(G_host) != len(self.shapes):
            raise ValueError(f"G_host: expected {len(self.shapes)} tensors, got {len(G_host)}")
        b = self._nfed & 1
        cs = self._copy_stream
        for used in (cs, s):  # the blocks stay allocated until these streams' work on them is done
            if used.cuda_stream not in self._buf_streams:
                self._buf_streams.add(used.cuda_stream)
                for d in self._gbuf[0] + self._gbuf[1]:
                    d.record_stream(used)
        with torch.cuda.stream(cs):
            if self._buf_free[b] is not None:
                cs.wait_event(self._buf_free[b])
            for d, h in zip(self._gbuf[b], G_host):
                if tuple(h.shape) != tuple(d.shape) or h.dtype != d.dtype:
                    raise ValueError(f"G_host: tensor {tuple(h.shape)} {h.dtype} does not match {tuple(d.shape)} "
                                     f"{d.dtype}")
                d.copy_(h, non_blocking=True)
            copied = torch.cuda.Event()
            copied.record(cs)
        s.wait_event(copied)
        self(W, self._gbuf[b], M, stream=s, **hp)
        done = torch.cuda.Event()
        done.record(s)
        self._buf_free[b] = done
        self._nfed += 1

    def host_copy_stream(self):
        """The side stream step_from_host copies on (created by its first call)."""
        return getattr(self, "_copy_stream", None)

    def momentum(self, G, state, U, beta=0.95, nesterov=True, seed=None, norms=None, stream=None) -> torch.Tensor:
        """The momentum of a step on a QuantizedState, by itself: the state updated in place, the blended direction
        in U, its Frobenius norms (one a matrix, fp32) returned.  G and U: the handle's dtype, stored by rows; U may be G."""
        s = self._on(stream)
        hp = B.make_hparams(0.0, beta, 0.0, 0.0, QUINTIC, nesterov, 0)
        g = _views(G, self._entries, self.device, "G", self.dtype, by_rows=True)
        u = _views(U, self._entries, self.device, "U", self.dtype, by_rows=True)
        if norms is not None:
            self._check_norms(norms)
        B.muon_momentum_state(self.handle, g, self._momentum_state(state), u, len(self.shapes), state._fmt, hp, seed, s)
        return self.norms(norms, stream=stream)

    def orthogonalize(self, X, O, eps=1e-7, abc=QUINTIC, ns_steps=None, stream=None):
        """O = the orthogonalised X, nothing else.

        In mode "half" X and O may be views stored by rows or by columns (slices, stacks, transposed tensors) of
        bf16, fp16 or fp32, O may be X itself, and abc may be a list with one coefficient triple per iteration.
        """
        if self.mode == "half":
            x = _views(X, self._entries, self.device, "X")
            o = _views(O, self._entries, self.device, "O")
            abc, ns_steps = self._coefficients(abc, ns_steps)
            hp = B.make_hparams(0.0, 0.0, 0.0, eps, abc, False, ns_steps)
            B.muon_orthogonalize_views(self.handle, x, o, len(self.shapes), hp, self._on(stream))
            return
        abc, ns_steps = self._coefficients(abc, ns_steps)
        hp = B.make_hparams(0.0, 0.0, 0.0, eps, abc, False, ns_steps)
        B.muon_orthogonalize(self.handle, self._check(X, "X"), self._check(O, "O"), hp, self._on(stream))

    def _check_norms(self, out):
        if out.dtype is not torch.float32 or out.numel() < self._n or not out.is_contiguous() or \
                out.device not in (self.device, torch.device("cpu")):
            raise ValueError(f"norms: tensor {tuple(out.shape)} {out.dtype} {out.device} is not {self._n} contiguous "
                             f"torch.float32 on {self.device} or the host")

    def norms(self, out=None, stream=None) -> torch.Tensor:
        """||U_i||_F of the last step, fp32, enqueued as one copy into `out` (device or pinned host)."""
        if out is not None:
            self._check_norms(out)
        elif stream is None:
            out = torch.empty(self._n, dtype=torch.float32, device=self.device)
        else:  # memory of the stream that writes it
            with torch.cuda.stream(stream):
                out = torch.empty(self._n, dtype=torch.float32, device=self.device)
        B.muon_get_norms(self.handle, out.data_ptr(), self._on(stream))
        return out

    def status(self, stream=None) -> int:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        return B.muon_get_status(self.handle, s.cuda_stream)

    def close(self):
        if getattr(self, "handle", None):
            B.muon_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0,
               stream=None):
    """AdamW on a list of tensors (bf16 or fp32 parameters, fp32 moments), one fused launch per 256 tensors.

    Every tensor must be contiguous and on the same CUDA device; `step` counts from 1.
    """
    if not params:
        return
    dt = params[0].dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError("parameters must be bf16 or fp32")
    for p, g, m, v in zip(params, grads, exp_avg, exp_avg_sq):
        if not (p.is_contiguous() and g.is_contiguous() and m.is_contiguous() and v.is_contiguous()):
            raise ValueError("tensors must be contiguous")
        if p.dtype != dt or g.dtype != dt or m.dtype != torch.float32 or v.dtype != torch.float32:
            raise ValueError("p, g share the parameter dtype; moments are fp32")
        if not (p.numel() == g.numel() == m.numel() == v.numel()):
            raise ValueError("p, g, m, v must have equal sizes")
    hp = B.AdamWHParams(float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step))
    s = stream if stream is not None else torch.cuda.current_stream(params[0].device)
    B.muon_adamw_step([p.data_ptr() for p in params], [g.data_ptr() for g in grads],
                      [m.data_ptr() for m in exp_avg], [v.data_ptr() for v in exp_avg_sq],
                      [p.numel() for p in params], B.MUON_BF16 if dt == torch.bfloat16 else B.MUON_FP32, hp,
                      s.cuda_stream)

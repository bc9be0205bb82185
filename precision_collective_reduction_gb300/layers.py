"""The operators around the collectives of a transformer layer, one Python
function per C entry point of that part of include/lpcoll.h, where their
semantics stand: the router (``expert_route``), tokens sorted by expert, sent
out as rows and brought back with their weights (``expert_sort``,
``expert_dispatch``, ``expert_combine``), the end of a block with its norms,
gate and residual (``residual_norm``), layer norms (``layer_norm``), the end of a
block with dropout (``residual_dropout``), the router's balance loss
(``expert_balance``), the rows of a vocabulary shard (``token_embed``), and the
gradients.

As in ``_binding``, the functions check the torch tensors they are given
(CUDA, on the current device, contiguous, of the right type and shape), pass
their pointers to the library and raise ``LpcollError`` on a non-zero status.
Results go into tensors that the caller provides; scratch memory is the
caller's ``workspace`` or, without one, torch's, on the call's stream (on the
default stream kept, at the largest call's size, until the thread ends; a caller
who wants the memory back passes a workspace).
"""
import contextlib
import ctypes
import operator
import threading
import warnings

from . import _binding as B

MAX_EXPERTS = 1024
MAX_TOPK = 32
MAX_HIDDEN = 16384
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3

_SORT_ONE_CTA = 2048  # slots that expert_sort takes without scratch memory
# host arrays of 0..16 device pointers
_POINTERS = [ctypes.c_void_p * n for n in range(B.MAX_RANKS + 1)]

torch = None  # imported by the first call, as everywhere in the binding
_raw_device = _raw_stream = None
_DTYPE = {}


def _device():
    """Index of the current CUDA device, which every call runs on."""
    global torch, _raw_device, _raw_stream
    if torch is None:
        t = B._torch()
        t.cuda.current_device()  # initializes CUDA, or says why not
        # the same without that check, and the current stream's handle without
        # a Stream object around it
        _raw_device = t._C._cuda_getDevice
        _raw_stream = t._C._cuda_getCurrentRawStream
        _DTYPE.update({t.float32: B.F32, t.bfloat16: B.BF16})
        torch = t
    return _raw_device()


def _ptr(t, what, dtype, shape, device, rank=None):
    """Device pointer of a tensor of that type, shape and device."""
    # the checks of a good tensor in as few calls as they take: at decode sizes
    # they cost more than the kernels
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if rank is not None:
        what = "%s[%d]" % (what, rank)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have the shape %s, got %s"
                         % (what, tuple(shape), tuple(t.shape)))
    if t.get_device() != device:  # -1 for a host tensor
        raise ValueError("%s must be a CUDA tensor of the current device cuda:%d, is on %s"
                         % (what, device, t.device))
    raise ValueError("%s must be contiguous" % what)


def _opt(t, what, dtype, shape, device):
    return None if t is None else _ptr(t, what, dtype, shape, device)


def _shape(t, dims, what):
    try:
        shape = t.shape
        if len(shape) == dims:
            return shape
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % what) from None
    raise ValueError("%s must have %d dimensions, got %s" % (what, dims, tuple(shape)))


def _code(t):
    code = _DTYPE.get(t.dtype)
    return B.dtype_code(t) if code is None else code


def _stream(stream, device):
    """cudaStream_t of the call; None is the current stream."""
    return _raw_stream(device) if stream is None else B._stream(stream)


# Scratch memory of each thread's calls on the default stream, by device. Calls
# of one thread on that stream run one after the other on the GPU, so they can
# share it; it grows to the largest call's need. (An allocation per call costs a
# small norm's gradient 6 of its 20 us.)
_scratch_of = threading.local()


def _scratch(workspace, need, stream, device):
    """(pointer, bytes, tensor) of the scratch memory of a call on cudaStream_t
    ``stream``. Memory of torch's allocator belongs to the stream it was taken
    on, so it cannot be given out again before the call's kernels are done."""
    if workspace is not None:
        n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
        p = _ptr(workspace, "workspace", torch.uint8, (n,), device)
        if n < need:
            raise ValueError("workspace holds %d bytes, needs %d" % (n, need))
        return p, n, workspace
    if need == 0:
        return None, 0, None
    if stream == 0:
        kept = _scratch_of.__dict__.get(device)
        if kept is None or kept[1] < need:
            t = _new_scratch(need, stream, device)
            kept = _scratch_of.__dict__[device] = (t.data_ptr(), need, t)
        return kept
    t = _new_scratch(need, stream, device)
    return t.data_ptr(), need, t


def _on(stream, device):
    """Context in which torch works on cudaStream_t ``stream``."""
    if stream == _raw_stream(device):
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if stream
                             else torch.cuda.default_stream())


def _new_scratch(need, stream, device):
    with _on(stream, device):
        return torch.empty(need, dtype=torch.uint8, device="cuda")


def _topk(ids, ntokens, what):
    T, K = _shape(ids, 2, what)
    if T != ntokens:
        raise ValueError("%s lists %d tokens, not %d" % (what, T, ntokens))
    return K


def expert_route(logits, ids, weights, renormalize=False, stream=None):
    """Router: the K largest of each token's logits [T, E] -> ids (int32
    [T, K], -1 where fewer than K experts are left) and weights (float32
    [T, K]): the softmax over all experts, or with ``renormalize`` over the
    chosen ones."""
    dev = _device()
    T, E = _shape(logits, 2, "logits")
    K = _topk(ids, T, "ids")
    lp = _ptr(logits, "logits", logits.dtype, (T, E), dev)
    ip = _ptr(ids, "ids", torch.int32, (T, K), dev)
    wp = _ptr(weights, "weights", torch.float32, (T, K), dev)
    B._check(B.lib().expert_route(lp, _code(logits), T, E, K, 1 if renormalize else 0, ip, wp,
                                  _stream(stream, dev)), "expert_route")
    return ids, weights


def expert_route_backward(logits, ids, weights, dweights, dlogits, renormalize=False,
                          stream=None):
    """dweights [T, K] -> dlogits [T, E], for ids and weights as expert_route
    wrote them with the same ``renormalize``."""
    dev = _device()
    T, E = _shape(logits, 2, "logits")
    K = _topk(ids, T, "ids")
    lp = _ptr(logits, "logits", logits.dtype, (T, E), dev)
    ip = _ptr(ids, "ids", torch.int32, (T, K), dev)
    wp = _ptr(weights, "weights", torch.float32, (T, K), dev)
    gp = _ptr(dweights, "dweights", torch.float32, (T, K), dev)
    op = _ptr(dlogits, "dlogits", logits.dtype, (T, E), dev)
    B._check(B.lib().expert_route_backward(lp, _code(logits), T, E, K, 1 if renormalize else 0,
                                           ip, wp, gp, op, _stream(stream, dev)),
             "expert_route_backward")
    return dlogits


def expert_sort_workspace_bytes(nslots, nexperts):
    """Scratch bytes of expert_sort (0 for a sort of one CTA)."""
    return B.lib().expert_sort_workspace_bytes(nslots, nexperts)


def expert_sort(ids, nexperts, slot_row, row_slot, offsets, counts, capacity=0,
                workspace=None, stream=None):
    """Stable sort of the slots of ids [T, K] by expert -> slot_row [T, K],
    row_slot [T * K] (or [nexperts * capacity]), offsets [nexperts + 1],
    counts [nexperts], all int32. capacity > 0 gives every expert that many
    rows, in equal chunks."""
    dev = _device()
    T, K = _shape(ids, 2, "ids")
    i32 = torch.int32
    capacity = int(capacity)
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    rows = nexperts * capacity if capacity else T * K
    p = (_ptr(ids, "ids", i32, (T, K), dev), _ptr(slot_row, "slot_row", i32, (T, K), dev),
         _ptr(row_slot, "row_slot", i32, (rows,), dev),
         _ptr(offsets, "offsets", i32, (nexperts + 1,), dev),
         _ptr(counts, "counts", i32, (nexperts,), dev))
    L = B.lib()
    need = L.expert_sort_workspace_bytes(T * K, nexperts) if T * K > _SORT_ONE_CTA else 0
    st = _stream(stream, dev)
    wp, wn, _keep = _scratch(workspace, need, st, dev)
    B._check(L.expert_sort(p[0], T * K, nexperts, capacity, p[1], p[2], p[3], p[4], wp, wn, st),
             "expert_sort")
    return slot_row, row_slot, offsets, counts


def _payload(codes, scales, R, H, dev):
    if codes is None or scales is None:
        raise ValueError("low precision (block=128) needs codes and scales")
    return (_ptr(codes, "codes", torch.uint8, (R, H), dev),
            _ptr(scales, "scales", torch.float32, (R, B.nblocks(H)), dev))


def expert_dispatch(x, slot_row, row_slot, out=None, block=0, codes=None, scales=None,
                    stream=None):
    """Tokens x [T, H] to rows sorted by expert: out [R, H], or with
    block=128 the FP8 payload codes (uint8 [R, H]) and scales (float32
    [R, ceil(H / 128)]) of each row. Rows without a slot are zeros."""
    dev = _device()
    T, H = _shape(x, 2, "x")
    K = _topk(slot_row, T, "slot_row")
    R, = _shape(row_slot, 1, "row_slot")
    xp = _ptr(x, "x", x.dtype, (T, H), dev)
    sp = _ptr(slot_row, "slot_row", torch.int32, (T, K), dev)
    rp = _ptr(row_slot, "row_slot", torch.int32, (R,), dev)
    op = cp = qp = None
    if block:
        cp, qp = _payload(codes, scales, R, H, dev)
    else:
        op = _ptr(out, "out", x.dtype, (R, H), dev)
    B._check(B.lib().expert_dispatch(xp, T, K, R, H, _code(x), block, sp, rp, op, cp, qp,
                                     _stream(stream, dev)), "expert_dispatch")
    return (codes, scales) if block else out


def expert_dispatch_backward(drows, slot_row, dx, stream=None):
    """Gradient of the exact expert_dispatch: dx[t] is the sum of the rows of
    token t's choices."""
    return expert_combine(slot_row, dx, drows, stream=stream)


def expert_combine(slot_row, out, rows=None, weights=None, block=0, codes=None, scales=None,
                   stream=None):
    """Rows [R, H] (with block=128 the payload codes, scales) back to their
    tokens: out[t] = sum_k weights[t, k] * rows[slot_row[t, k]]; weights None
    stands for 1."""
    dev = _device()
    T, H = _shape(out, 2, "out")
    K = _topk(slot_row, T, "slot_row")
    op = _ptr(out, "out", out.dtype, (T, H), dev)
    sp = _ptr(slot_row, "slot_row", torch.int32, (T, K), dev)
    rp = cp = qp = None
    if block:
        R = _shape(codes, 2, "codes")[0] if codes is not None else 0
        cp, qp = _payload(codes, scales, R, H, dev)
    else:
        R = _shape(rows, 2, "rows")[0]
        rp = _ptr(rows, "rows", out.dtype, (R, H), dev)
    wp = _opt(weights, "weights", torch.float32, (T, K), dev)
    B._check(B.lib().expert_combine(rp, cp, qp, T, K, R, H, _code(out), block, sp, wp, op,
                                    _stream(stream, dev)), "expert_combine")
    return out


def expert_combine_backward(dout, slot_row, row_slot, drows, rows=None, weights=None,
                            dweights=None, stream=None):
    """dout [T, H] -> drows [R, H] and, if given, dweights [T, K] (which needs
    the rows that were combined)."""
    dev = _device()
    T, H = _shape(dout, 2, "dout")
    K = _topk(slot_row, T, "slot_row")
    R, = _shape(row_slot, 1, "row_slot")
    dt = dout.dtype
    if dweights is not None and rows is None:
        raise ValueError("dweights needs rows")
    p = (_ptr(dout, "dout", dt, (T, H), dev), _opt(rows, "rows", dt, (R, H), dev),
         _ptr(slot_row, "slot_row", torch.int32, (T, K), dev),
         _ptr(row_slot, "row_slot", torch.int32, (R,), dev),
         _opt(weights, "weights", torch.float32, (T, K), dev),
         _ptr(drows, "drows", dt, (R, H), dev),
         _opt(dweights, "dweights", torch.float32, (T, K), dev))
    B._check(B.lib().expert_combine_backward(p[0], p[1], T, K, R, H, _code(dout), p[2], p[3],
                                             p[4], p[5], p[6], _stream(stream, dev)),
             "expert_combine_backward")
    return drows, dweights


def _gate(gate, dtype, T, H, dev, kind):
    """(kind, pointer) of a gate of shape [H], [T] or [T, H]. A gate of one
    dimension is one value per channel if it has H values, whatever T is;
    ``kind`` says otherwise. Where both fit and differ, so that a caller's gate
    per token would change its meaning with the batch, a warning asks for it."""
    if gate is None:
        return GATE_NONE, None
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if kind is None:
        kind = "full" if gate.dim() == 2 else "channel" if gate.shape == (H,) else "token"
        if kind == "channel" and T == H > 1:
            warnings.warn("gate of %d values for as many tokens as channels is taken as one per "
                          "channel: say so, or otherwise, with gate_kind" % H, stacklevel=3)
    if kind not in ("channel", "token", "full"):
        raise ValueError("gate_kind must be 'channel', 'token' or 'full', got %r" % (kind,))
    shape = {"channel": (H,), "token": (T,), "full": (T, H)}[kind]
    code = {"channel": GATE_CHANNEL, "token": GATE_TOKEN, "full": GATE_FULL}[kind]
    return code, _ptr(gate, "gate", dtype, shape, dev)


def residual_norm(h, x, x_out, n_out=None, gate=None, w_post=None, w_pre=None, res_scale=1.0,
                  branch_scale=1.0, eps=1e-6, h_sum=None, gate_kind=None, stream=None):
    """End of a block: h (one [T, H] tensor, or the partial products of up to
    16 ranks) is summed and, with ``w_post`` [H], RMS-normed, gated (``gate``
    [H], [T] or [T, H]) and added to the residual x: x_out = res_scale * x +
    branch_scale * gate * u. With ``w_pre`` [H], n_out is the RMS norm of
    x_out. ``h_sum`` receives the summed h. ``gate_kind`` ("channel", "token",
    "full") names the gate's kind; without it the shape does, and [H] goes
    before [T] where the two are equal, with a warning."""
    dev = _device()
    if isinstance(h, torch.Tensor):
        h = (h,)
    T, H = _shape(x, 2, "x")
    dt = x.dtype
    hp = [_ptr(t, "h", dt, (T, H), dev, r) for r, t in enumerate(h)]
    if not 1 <= len(hp) <= B.MAX_RANKS:
        raise ValueError("need 1 to %d ranks, got %d" % (B.MAX_RANKS, len(hp)))
    kind, gp = _gate(gate, dt, T, H, dev, gate_kind)
    if w_pre is not None and n_out is None:
        raise ValueError("w_pre needs n_out")
    xp = _ptr(x, "x", dt, (T, H), dev)
    post = _opt(w_post, "w_post", dt, (H,), dev)
    pre = _opt(w_pre, "w_pre", dt, (H,), dev)
    op = _ptr(x_out, "x_out", dt, (T, H), dev)
    np_ = _ptr(n_out, "n_out", dt, (T, H), dev) if w_pre is not None else None
    sp = _opt(h_sum, "h_sum", dt, (T, H), dev)
    B._check(B.lib().residual_norm(_POINTERS[len(hp)](*hp), len(hp), xp, gp, kind, post, pre, res_scale,
                                   branch_scale, eps, T, H, _code(x), op, np_, sp,
                                   _stream(stream, dev)), "residual_norm")
    return x_out, n_out


def residual_norm_backward_workspace_bytes(ntokens, hidden, dtype):
    """Scratch bytes of residual_norm_backward; dtype F32 or BF16."""
    return B.lib().residual_norm_backward_workspace_bytes(ntokens, hidden, dtype)


def residual_norm_backward(dx_out, dn_out, h, x_out, dx, dh, gate=None, w_post=None, w_pre=None,
                           res_scale=1.0, branch_scale=1.0, eps=1e-6, dgate=None, dw_post=None,
                           dw_pre=None, gate_kind=None, workspace=None, stream=None):
    """Gradients of residual_norm: dx_out, dn_out (either may be None where
    that output has no gradient or does not exist), the summed h and the
    result x_out -> dx, dh and, where given, dgate (float32 [H] or [T], or of
    x_out's type [T, H]), dw_post and dw_pre (float32 [H]). Without dn_out,
    dw_pre is zeros."""
    dev = _device()
    T, H = _shape(x_out, 2, "x_out")
    dt, f32 = x_out.dtype, torch.float32
    kind, gp = _gate(gate, dt, T, H, dev, gate_kind)
    for g, w, what in ((dgate, gate, "gate"), (dw_post, w_post, "w_post"),
                       (dw_pre, w_pre, "w_pre")):
        if g is not None and w is None:
            raise ValueError("a gradient of %s needs %s" % (what, what))
    if dx_out is None and dn_out is None:
        raise ValueError("need dx_out or dn_out")
    if dn_out is not None and w_pre is None:
        raise ValueError("dn_out needs w_pre")
    gshape = {GATE_CHANNEL: (H,), GATE_TOKEN: (T,), GATE_FULL: (T, H)}.get(kind)
    p = (_opt(dx_out, "dx_out", dt, (T, H), dev), _opt(dn_out, "dn_out", dt, (T, H), dev),
         _ptr(h, "h", dt, (T, H), dev), _ptr(x_out, "x_out", dt, (T, H), dev))
    post = _opt(w_post, "w_post", dt, (H,), dev)
    pre = _opt(w_pre, "w_pre", dt, (H,), dev)
    q = (_ptr(dx, "dx", dt, (T, H), dev), _ptr(dh, "dh", dt, (T, H), dev),
         _opt(dgate, "dgate", dt if kind == GATE_FULL else f32, gshape, dev),
         _opt(dw_post, "dw_post", f32, (H,), dev), _opt(dw_pre, "dw_pre", f32, (H,), dev))
    L = B.lib()
    code = _code(x_out)
    need = L.residual_norm_backward_workspace_bytes(T, H, code)
    st = _stream(stream, dev)
    if dn_out is None:  # the second norm has no part in these gradients
        pre = None
    wp, wn, _keep = _scratch(workspace, need, st, dev)
    B._check(L.residual_norm_backward(p[0], p[1], p[2], p[3], gp, kind, post, pre, res_scale,
                                      branch_scale, eps, T, H, code, q[0], q[1], q[2], q[3],
                                      q[4], wp, wn, st),
             "residual_norm_backward")
    if dn_out is None and dw_pre is not None:
        with _on(st, dev):
            dw_pre.detach().zero_()
    return dx, dh


def _rows_of(h):
    return (h,) if isinstance(h, torch.Tensor) else h


def layer_norm(x, out, w=None, b=None, eps=1e-5, stream=None):
    """Layer norm of the rows of x [T, H]: out = (x - mean) / sqrt(var + eps) *
    w + b, with w, b [H] (None stands for ones and zeros)."""
    dev = _device()
    T, H = _shape(x, 2, "x")
    dt = x.dtype
    p = (_ptr(x, "x", dt, (T, H), dev), _opt(w, "w", dt, (H,), dev), _opt(b, "b", dt, (H,), dev),
         _ptr(out, "out", dt, (T, H), dev))
    B._check(B.lib().layer_norm(p[0], p[1], p[2], eps, T, H, _code(x), p[3],
                                _stream(stream, dev)), "layer_norm")
    return out


def layer_norm_backward_workspace_bytes(ntokens, hidden, dtype):
    """Scratch bytes of layer_norm_backward; dtype F32 or BF16."""
    return B.lib().layer_norm_backward_workspace_bytes(ntokens, hidden, dtype)


def layer_norm_backward(dout, x, dx=None, w=None, eps=1e-5, dw=None, db=None, workspace=None,
                        stream=None):
    """Gradients of layer_norm: dout and its input x -> dx and, where given, dw
    and db (float32 [H])."""
    dev = _device()
    T, H = _shape(x, 2, "x")
    dt, f32 = x.dtype, torch.float32
    p = (_ptr(dout, "dout", dt, (T, H), dev), _ptr(x, "x", dt, (T, H), dev),
         _opt(w, "w", dt, (H,), dev), _opt(dx, "dx", dt, (T, H), dev),
         _opt(dw, "dw", f32, (H,), dev), _opt(db, "db", f32, (H,), dev))
    L = B.lib()
    code = _code(x)
    sums = dw is not None or db is not None
    need = L.layer_norm_backward_workspace_bytes(T, H, code) if sums else 0
    st = _stream(stream, dev)
    wp, wn, _keep = _scratch(workspace, need, st, dev)
    B._check(L.layer_norm_backward(p[0], p[1], p[2], eps, T, H, code, p[3], p[4], p[5], wp, wn,
                                   st), "layer_norm_backward")
    return dx


def residual_dropout(h, x, x_out, rng, p, n_out=None, w=None, b=None, eps=1e-5, first_row=0,
                     stream=None):
    """End of a block of a model with layer norms: h (one [T, H] tensor, or the
    partial products of up to 16 ranks) is summed, dropped with probability p
    (what stays is divided by 1 - p) and added to the residual x (or None):
    x_out. With ``n_out``, the layer norm of x_out (w, b, eps). ``rng``: int64
    [2] on the GPU, seed and offset (as 64 bits), read when the kernel runs; may
    be None if p is 0. ``first_row`` numbers the rows of a part of a larger
    batch."""
    dev = _device()
    h = _rows_of(h)
    T, H = _shape(x_out, 2, "x_out")
    dt = x_out.dtype
    hp = [_ptr(t, "h", dt, (T, H), dev, r) for r, t in enumerate(h)]
    if not 1 <= len(hp) <= B.MAX_RANKS:
        raise ValueError("need 1 to %d ranks, got %d" % (B.MAX_RANKS, len(hp)))
    if n_out is None and (w is not None or b is not None):
        raise ValueError("w and b need n_out")
    q = (_opt(x, "x", dt, (T, H), dev), _opt(rng, "rng", torch.int64, (2,), dev),
         _opt(w, "w", dt, (H,), dev), _opt(b, "b", dt, (H,), dev),
         _ptr(x_out, "x_out", dt, (T, H), dev), _opt(n_out, "n_out", dt, (T, H), dev))
    B._check(B.lib().residual_dropout(_POINTERS[len(hp)](*hp), len(hp), q[0], q[1], p,
                                      _row_number(first_row), q[2], q[3], eps, T, H,
                                      _code(x_out), q[4], q[5], _stream(stream, dev)),
             "residual_dropout")
    return x_out, n_out


def _row_number(first_row):
    if first_row < 0:
        raise ValueError("first_row must not be negative")
    return first_row


def residual_dropout_backward_workspace_bytes(ntokens, hidden, dtype):
    """Scratch bytes of residual_dropout_backward; dtype F32 or BF16."""
    return B.lib().residual_dropout_backward_workspace_bytes(ntokens, hidden, dtype)


def residual_dropout_backward(dx_out, dn_out, x_out, dx, dh, rng, p, w=None, eps=1e-5, dw=None,
                              db=None, first_row=0, workspace=None, stream=None):
    """Gradients of residual_dropout: dx_out, dn_out (either may be None where that
    output has no gradient or does not exist) and, with dn_out, the result x_out
    -> dx (or None), dh (or None) and, where given, dw and db (float32 [H]; zeros
    without dn_out). rng, p and first_row are the forward pass's."""
    dev = _device()
    like = dn_out if dn_out is not None else dx_out
    if like is None:
        raise ValueError("need dx_out or dn_out")
    T, H = _shape(like, 2, "dn_out" if dn_out is not None else "dx_out")
    dt, f32 = like.dtype, torch.float32
    if dn_out is not None and x_out is None:
        raise ValueError("dn_out needs x_out")
    q = (_opt(dx_out, "dx_out", dt, (T, H), dev), _opt(dn_out, "dn_out", dt, (T, H), dev),
         _opt(x_out, "x_out", dt, (T, H), dev), _opt(rng, "rng", torch.int64, (2,), dev),
         _opt(w, "w", dt, (H,), dev), _opt(dx, "dx", dt, (T, H), dev),
         _opt(dh, "dh", dt, (T, H), dev), _opt(dw, "dw", f32, (H,), dev),
         _opt(db, "db", f32, (H,), dev))
    L = B.lib()
    code = _code(like)
    need = 0
    if dn_out is not None and (dw is not None or db is not None):
        need = L.residual_dropout_backward_workspace_bytes(T, H, code)
    st = _stream(stream, dev)
    wp, wn, _keep = _scratch(workspace, need, st, dev)
    B._check(L.residual_dropout_backward(q[0], q[1], q[2], q[3], p, _row_number(first_row), q[4],
                                         eps, T, H, code, q[5], q[6], q[7], q[8], wp, wn, st),
             "residual_dropout_backward")
    return dx, dh


def _valid(valid, ntokens, dev):
    if valid is not None and isinstance(valid, torch.Tensor) and valid.dtype == torch.bool:
        return _ptr(valid, "valid", torch.bool, (ntokens,), dev)
    return _opt(valid, "valid", torch.uint8, (ntokens,), dev)


def expert_balance_workspace_bytes(ntokens, nexperts):
    """Scratch bytes of expert_balance."""
    return B.lib().expert_balance_workspace_bytes(ntokens, nexperts)


def expert_balance(logits, ids, loss, counts, prob_sums, coef=1.0, valid=None, workspace=None,
                   stream=None):
    """Balance loss of a router: logits [T, E] and the ids [T, K] that
    expert_route chose -> loss (float32 [1]), counts (int32 [E + 1]: choices of
    every expert, then the valid tokens) and prob_sums (float32 [E], the sums of
    the softmax). ``valid`` (uint8 or bool [T]) is 0 where a token is padding."""
    dev = _device()
    T, E = _shape(logits, 2, "logits")
    K = _topk(ids, T, "ids")
    f32, i32 = torch.float32, torch.int32
    p = (_ptr(logits, "logits", logits.dtype, (T, E), dev), _ptr(ids, "ids", i32, (T, K), dev),
         _valid(valid, T, dev), _ptr(loss, "loss", f32, (1,), dev),
         _ptr(counts, "counts", i32, (E + 1,), dev), _ptr(prob_sums, "prob_sums", f32, (E,), dev))
    L = B.lib()
    st = _stream(stream, dev)
    wp, wn, _keep = _scratch(workspace, L.expert_balance_workspace_bytes(T, E), st, dev)
    B._check(L.expert_balance(p[0], _code(logits), T, E, p[1], K, p[2], coef, p[3], p[4], p[5],
                              wp, wn, st), "expert_balance")
    return loss


def expert_balance_backward(logits, counts, dloss, dlogits, coef=1.0, valid=None,
                            accumulate=False, stream=None):
    """dloss (float32 [1]) -> dlogits [T, E], for the counts that expert_balance
    wrote (or their sums over ranks) and the same coef and valid. With
    ``accumulate`` the gradient is added to dlogits, say to
    expert_route_backward's."""
    dev = _device()
    T, E = _shape(logits, 2, "logits")
    dt = logits.dtype
    p = (_ptr(logits, "logits", dt, (T, E), dev), _valid(valid, T, dev),
         _ptr(counts, "counts", torch.int32, (E + 1,), dev),
         _ptr(dloss, "dloss", torch.float32, (1,), dev),
         _ptr(dlogits, "dlogits", dt, (T, E), dev))
    B._check(B.lib().expert_balance_backward(p[0], _code(logits), T, E, p[1], p[2], coef, p[3],
                                             1 if accumulate else 0, p[4], _stream(stream, dev)),
             "expert_balance_backward")
    return dlogits


def _ids(ids, dev):
    """(pointer, type code, tokens) of the token ids, int32 or int64 [T]."""
    T, = _shape(ids, 1, "ids")
    if ids.dtype == torch.int64:
        return _ptr(ids, "ids", torch.int64, (T,), dev), 1, T
    return _ptr(ids, "ids", torch.int32, (T,), dev), 0, T


def _first_id(first_id):
    # ctypes would take it modulo 2^64, where it stands for other ids
    first_id = operator.index(first_id)
    if not -(1 << 63) <= first_id < 1 << 63:
        raise ValueError("first_id must be a 64-bit number")
    return first_id


def token_embed(table, ids, out, first_id=0, scale=1.0, stream=None):
    """Rows of a shard of a vocabulary: table [V, H] holds the ids first_id ..
    first_id + V - 1; out [T, H] = scale * table[ids - first_id], and zeros for
    all other ids (int32 or int64 [T])."""
    dev = _device()
    ip, index, T = _ids(ids, dev)
    V, H = _shape(table, 2, "table")
    tp = _ptr(table, "table", table.dtype, (V, H), dev)
    op = _ptr(out, "out", table.dtype, (T, H), dev)
    B._check(B.lib().token_embed(tp, V, ip, index, _first_id(first_id), T, H, _code(table), scale,
                                 op, _stream(stream, dev)), "token_embed")
    return out


def token_embed_backward_workspace_bytes(ntokens, vocab, hidden):
    """Scratch bytes of token_embed_backward."""
    return B.lib().token_embed_backward_workspace_bytes(ntokens, vocab, hidden)


def token_embed_backward(dout, ids, dtable, first_id=0, scale=1.0, accumulate=False,
                         workspace=None, stream=None):
    """dout [T, H] -> dtable (float32 [V, H]): every row the scaled sum of its
    tokens' gradients, zeros in rows without a token. With ``accumulate`` the
    sums are added to dtable, and rows without a token are not touched."""
    dev = _device()
    ip, index, T = _ids(ids, dev)
    V, H = _shape(dtable, 2, "dtable")
    gp = _ptr(dout, "dout", dout.dtype if isinstance(dout, torch.Tensor) else None, (T, H), dev)
    tp = _ptr(dtable, "dtable", torch.float32, (V, H), dev)
    L = B.lib()
    st = _stream(stream, dev)
    need = L.token_embed_backward_workspace_bytes(T, V, H)
    wp, wn, _keep = _scratch(workspace, need, st, dev)
    B._check(L.token_embed_backward(gp, ip, index, _first_id(first_id), T, V, H, _code(dout),
                                    scale, 1 if accumulate else 0, tp, wp, wn, st),
             "token_embed_backward")
    return dtable

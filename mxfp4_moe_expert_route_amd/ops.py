"""Torch-tensor wrappers with the C ABI's names (argument marshalling only).

Each wrapper checks device, dtype, shape and contiguity, allocates outputs
that were not passed in, and calls the library on the current HIP stream.
Every step of the computation runs in libmxfp4moe.so."""

import torch

from ._lib import check, lib

F32, BF16 = 0, 1


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _need(t, name, dtype, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _need(t, name, dtype, shape, device)


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() else None


# ---------------------------------------------------------------------------

def mxfp4_pack(x, codes=None, scales=None):
    """x [rows, K] float32 or bfloat16 -> (codes uint8 [rows, K/2], scales uint8 [rows, K/32])."""
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be float32 or bfloat16")
    _need(x, "x", x.dtype)
    rows, K = x.shape
    codes = _out(codes, "codes", torch.uint8, (rows, K // 2), x.device)
    scales = _out(scales, "scales", torch.uint8, (rows, K // 32), x.device)
    check(lib().mxfp4_pack(_ptr(x), BF16 if x.dtype == torch.bfloat16 else F32, rows, K,
                           _ptr(codes), _ptr(scales), _stream()), "mxfp4_pack")
    return codes, scales


def mxfp4_unpack(codes, scales, dtype=torch.float32, out=None):
    """(codes [rows, K/2], scales [rows, K/32]) -> [rows, K] float32 or bfloat16."""
    _need(codes, "codes", torch.uint8)
    rows, half = codes.shape
    K = 2 * half
    _need(scales, "scales", torch.uint8, (rows, K // 32), codes.device)
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dtype must be float32 or bfloat16")
    out = _out(out, "out", dtype, (rows, K), codes.device)
    check(lib().mxfp4_unpack(_ptr(codes), _ptr(scales), rows, K, _ptr(out),
                             BF16 if dtype == torch.bfloat16 else F32, _stream()), "mxfp4_unpack")
    return out


def moe_route_topk(logits, k, topk_ids=None, topk_w=None):
    """logits [T, E] float32 -> (ids int32 [T, k], weights float32 [T, k])."""
    _need(logits, "logits", torch.float32)
    T, E = logits.shape
    topk_ids = _out(topk_ids, "topk_ids", torch.int32, (T, k), logits.device)
    topk_w = _out(topk_w, "topk_w", torch.float32, (T, k), logits.device)
    check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream()),
          "moe_route_topk")
    return topk_ids, topk_w


def moe_router_topk(x, w_router, k, bias=None, logits=None, topk_ids=None, topk_w=None):
    """x [T, H] bfloat16, w_router [E, H] float32 (bias [E] float32 or None)
    -> (logits float32 [T, E], ids int32 [T, k], weights float32 [T, k])."""
    _need(x, "x", torch.bfloat16)
    _need(w_router, "w_router", torch.float32)
    T, H = x.shape
    E, H2 = w_router.shape
    if H2 != H:
        raise ValueError("w_router must be [E, H] with H = x.shape[1]")
    if bias is not None:
        _need(bias, "bias", torch.float32)
        if tuple(bias.shape) != (E,):
            raise ValueError("bias must be [E]")
    logits = _out(logits, "logits", torch.float32, (T, E), x.device)
    topk_ids = _out(topk_ids, "topk_ids", torch.int32, (T, k), x.device)
    topk_w = _out(topk_w, "topk_w", torch.float32, (T, k), x.device)
    check(lib().moe_router_topk(_ptr(x), _ptr(w_router), _ptr(bias) if bias is not None else None,
                                T, H, E, k, _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
                                _stream()), "moe_router_topk")
    return logits, topk_ids, topk_w


def dflash_verify_accept(target_logits, draft_probs, draft_tokens, uniforms, accept_len=None,
                         next_token=None, workspace=None):
    """target_logits [B, L+1, V] f32, draft_probs [B, L, V] f32, draft_tokens
    [B, L] int32, uniforms [B, L+1] f32 -> (accept_len int32 [B], next_token
    int32 [B])."""
    _need(target_logits, "target_logits", torch.float32)
    _need(draft_probs, "draft_probs", torch.float32)
    _need(draft_tokens, "draft_tokens", torch.int32)
    _need(uniforms, "uniforms", torch.float32)
    B, L1, V = target_logits.shape
    L = L1 - 1
    if tuple(draft_probs.shape) != (B, L, V) or tuple(draft_tokens.shape) != (B, L) or \
            tuple(uniforms.shape) != (B, L + 1):
        raise ValueError("shapes must be [B, L+1, V], [B, L, V], [B, L], [B, L+1]")
    dev = target_logits.device
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    next_token = _out(next_token, "next_token", torch.int32, (B,), dev)
    nbytes = int(lib().dflash_verify_workspace_bytes(B, L, V))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 8), dtype=torch.uint8, device=dev)
    check(lib().dflash_verify_accept(_ptr(target_logits), _ptr(draft_probs), _ptr(draft_tokens),
                                     _ptr(uniforms), B, L, V, _ptr(accept_len), _ptr(next_token),
                                     _ptr(workspace), workspace.numel(), _stream()),
          "dflash_verify_accept")
    return accept_len, next_token


def moe_permute_workspace_bytes(T, E, k):
    return int(lib().moe_permute_workspace_bytes(T, E, k))


def moe_permute(topk_ids, E, counts=None, offsets=None, sorted_pairs=None, pair_to_row=None,
                workspace=None):
    """topk_ids [T, k] int32 -> (counts [E], offsets [E+1], sorted_pairs [T*k], pair_to_row [T*k])."""
    _need(topk_ids, "topk_ids", torch.int32)
    T, k = topk_ids.shape
    dev = topk_ids.device
    counts = _out(counts, "counts", torch.int32, (E,), dev)
    offsets = _out(offsets, "offsets", torch.int32, (E + 1,), dev)
    sorted_pairs = _out(sorted_pairs, "sorted_pairs", torch.int32, (T * k,), dev)
    pair_to_row = _out(pair_to_row, "pair_to_row", torch.int32, (T * k,), dev)
    nws = moe_permute_workspace_bytes(T, E, k)
    if workspace is None and nws:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
    wsb = workspace.numel() if workspace is not None else 0
    check(lib().moe_permute(_ptr(topk_ids), T, E, k, _ptr(counts), _ptr(offsets),
                            _ptr(sorted_pairs), _ptr(pair_to_row), _ptr(workspace), wsb,
                            _stream()), "moe_permute")
    return counts, offsets, sorted_pairs, pair_to_row


def moe_route_permute(logits, k, topk_ids=None, topk_w=None, counts=None, offsets=None,
                      sorted_pairs=None, pair_to_row=None, workspace=None):
    """logits [T, E] f32 -> (topk_ids [T, k], topk_w [T, k], counts [E], offsets [E+1],
    sorted_pairs [T*k], pair_to_row [T*k]); moe_route_topk then moe_permute in one call."""
    _need(logits, "logits", torch.float32)
    T, E = logits.shape
    dev = logits.device
    topk_ids = _out(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    topk_w = _out(topk_w, "topk_w", torch.float32, (T, k), dev)
    counts = _out(counts, "counts", torch.int32, (E,), dev)
    offsets = _out(offsets, "offsets", torch.int32, (E + 1,), dev)
    sorted_pairs = _out(sorted_pairs, "sorted_pairs", torch.int32, (T * k,), dev)
    pair_to_row = _out(pair_to_row, "pair_to_row", torch.int32, (T * k,), dev)
    nws = moe_permute_workspace_bytes(T, E, k)
    if workspace is None and nws:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
    wsb = workspace.numel() if workspace is not None else 0
    check(lib().moe_route_permute(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w),
                                  _ptr(counts), _ptr(offsets), _ptr(sorted_pairs),
                                  _ptr(pair_to_row), _ptr(workspace), wsb, _stream()),
          "moe_route_permute")
    return topk_ids, topk_w, counts, offsets, sorted_pairs, pair_to_row


def moe_mxfp4_gate_up_swiglu(x, sorted_pairs, offsets, k, w13_codes, w13_scales, h=None):
    """x [T, H] bf16 -> h [T*k, I] bf16 (rows in sorted order)."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    E, two_i, half_h = w13_codes.shape
    I = two_i // 2
    dev = x.device
    _need(sorted_pairs, "sorted_pairs", torch.int32, (T * k,), dev)
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _need(w13_codes, "w13_codes", torch.uint8, (E, 2 * I, H // 2), dev)
    _need(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32), dev)
    h = _out(h, "h", torch.bfloat16, (T * k, I), dev)
    check(lib().moe_mxfp4_gate_up_swiglu(_ptr(x), _ptr(sorted_pairs), _ptr(offsets), T, H, I, E,
                                         k, _ptr(w13_codes), _ptr(w13_scales), _ptr(h),
                                         _stream()), "moe_mxfp4_gate_up_swiglu")
    return h


def moe_mxfp4_down(h, offsets, k, w2_codes, w2_scales, y=None):
    """h [T*k, I] bf16 -> y [T*k, H] float32 (rows in sorted order)."""
    _need(h, "h", torch.bfloat16)
    R, I = h.shape
    T = R // k
    E, H, _ = w2_codes.shape
    dev = h.device
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    _need(w2_codes, "w2_codes", torch.uint8, (E, H, I // 2), dev)
    _need(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32), dev)
    y = _out(y, "y", torch.float32, (R, H), dev)
    check(lib().moe_mxfp4_down(_ptr(h), _ptr(offsets), T, H, I, E, k, _ptr(w2_codes),
                               _ptr(w2_scales), _ptr(y), _stream()), "moe_mxfp4_down")
    return y


def moe_combine(y, topk_w, pair_to_row, out=None):
    """y [T*k, H] float32, topk_w [T, k] -> out [T, H] float32."""
    _need(topk_w, "topk_w", torch.float32)
    T, k = topk_w.shape
    _need(y, "y", torch.float32)
    H = y.shape[1]
    dev = y.device
    _need(y, "y", torch.float32, (T * k, H), dev)
    _need(pair_to_row, "pair_to_row", torch.int32, (T * k,), dev)
    out = _out(out, "out", torch.float32, (T, H), dev)
    check(lib().moe_combine(_ptr(y), _ptr(topk_w), _ptr(pair_to_row), T, H, k, _ptr(out),
                            _stream()), "moe_combine")
    return out


class LayerBuffers:
    """Preallocated intermediates of one layer call (so a timed loop allocates nothing)."""

    def __init__(self, T, H, I, E, k, device):
        R = T * k
        z = dict(device=device)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, **z)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, **z)
        self.counts = torch.empty((E,), dtype=torch.int32, **z)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, **z)
        self.sorted_pairs = torch.empty((R,), dtype=torch.int32, **z)
        self.pair_to_row = torch.empty((R,), dtype=torch.int32, **z)
        self.h = torch.empty((R, I), dtype=torch.bfloat16, **z)
        self.y = torch.empty((R, H), dtype=torch.float32, **z)
        self.out = torch.empty((T, H), dtype=torch.float32, **z)
        nws = moe_permute_workspace_bytes(T, E, k)
        self.workspace = torch.empty(max(nws, 1), dtype=torch.uint8, **z)


def moe_mxfp4_layer(x, logits, k, w13_codes, w13_scales, w2_codes, w2_scales, buffers=None):
    """Whole layer in one C call (route, permute, gate/up, down, combine).

    Returns the LayerBuffers holding every intermediate; `.out` is the result."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    E, two_i, _ = w13_codes.shape
    I = two_i // 2
    dev = x.device
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(w13_codes, "w13_codes", torch.uint8, (E, 2 * I, H // 2), dev)
    _need(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32), dev)
    _need(w2_codes, "w2_codes", torch.uint8, (E, H, I // 2), dev)
    _need(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32), dev)
    b = buffers if buffers is not None else LayerBuffers(T, H, I, E, k, dev)
    if (b.T, b.H, b.I, b.E, b.k) != (T, H, I, E, k):
        raise ValueError("buffers were made for another shape")
    check(lib().moe_mxfp4_layer(
        _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
        _ptr(w2_scales), _ptr(b.topk_ids), _ptr(b.topk_w), _ptr(b.counts), _ptr(b.offsets),
        _ptr(b.sorted_pairs), _ptr(b.pair_to_row), _ptr(b.h), _ptr(b.y), _ptr(b.out),
        _ptr(b.workspace), b.workspace.numel(), _stream()), "moe_mxfp4_layer")
    return b


def moe_mxfp4_decode_layer_workspace_bytes(T, H, I, E, k):
    """Bytes of the zero-filled workspace moe_mxfp4_decode_layer needs (0: the
    persistent kernel does not take these sizes)."""
    return int(lib().moe_mxfp4_decode_layer_workspace_bytes(T, H, I, E, k))


def decode_layer_workspace(T, H, I, E, k, device):
    """A zero-filled workspace for moe_mxfp4_decode_layer (None if the sizes
    are not taken).  Each call leaves it zero-filled, so it is reusable."""
    n = moe_mxfp4_decode_layer_workspace_bytes(T, H, I, E, k)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def moe_mxfp4_decode_layer(x, logits, k, w13_codes, w13_scales, w2_codes, w2_scales, workspace,
                           buffers=None):
    """The whole layer as one persistent kernel (verify-sized batches, T <= 16).

    `workspace` comes from decode_layer_workspace (zero-filled; the call leaves
    it so).  Returns the LayerBuffers holding every intermediate; `.out` is the
    result, equal bit for bit to moe_mxfp4_layer's."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    E, two_i, _ = w13_codes.shape
    I = two_i // 2
    dev = x.device
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(w13_codes, "w13_codes", torch.uint8, (E, 2 * I, H // 2), dev)
    _need(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32), dev)
    _need(w2_codes, "w2_codes", torch.uint8, (E, H, I // 2), dev)
    _need(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    b = buffers if buffers is not None else LayerBuffers(T, H, I, E, k, dev)
    if (b.T, b.H, b.I, b.E, b.k) != (T, H, I, E, k):
        raise ValueError("buffers were made for another shape")
    check(lib().moe_mxfp4_decode_layer(
        _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
        _ptr(w2_scales), _ptr(b.topk_ids), _ptr(b.topk_w), _ptr(b.counts), _ptr(b.offsets),
        _ptr(b.sorted_pairs), _ptr(b.pair_to_row), _ptr(b.h), _ptr(b.y), _ptr(b.out),
        _ptr(workspace), workspace.numel(), _stream()), "moe_mxfp4_decode_layer")
    return b


def moe_mxfp4_layer_noalloc(x, logits, k, w13_codes, w13_scales, w2_codes, w2_scales, buffers):
    """moe_mxfp4_layer through the entry point that allocates nothing: its
    grouping workspace is the library's fixed device scratch (the workspace
    tensor of `buffers` is not used).  `buffers` (LayerBuffers of this shape)
    must be passed in, so the call itself allocates nothing either."""
    _need(x, "x", torch.bfloat16)
    T, H = x.shape
    E, two_i, _ = w13_codes.shape
    I = two_i // 2
    dev = x.device
    _need(logits, "logits", torch.float32, (T, E), dev)
    _need(w13_codes, "w13_codes", torch.uint8, (E, 2 * I, H // 2), dev)
    _need(w13_scales, "w13_scales", torch.uint8, (E, 2 * I, H // 32), dev)
    _need(w2_codes, "w2_codes", torch.uint8, (E, H, I // 2), dev)
    _need(w2_scales, "w2_scales", torch.uint8, (E, H, I // 32), dev)
    b = buffers
    if (b.T, b.H, b.I, b.E, b.k) != (T, H, I, E, k):
        raise ValueError("buffers were made for another shape")
    check(lib().moe_mxfp4_layer_noalloc(
        _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
        _ptr(w2_scales), _ptr(b.topk_ids), _ptr(b.topk_w), _ptr(b.counts), _ptr(b.offsets),
        _ptr(b.sorted_pairs), _ptr(b.pair_to_row), _ptr(b.h), _ptr(b.y), _ptr(b.out),
        _stream()), "moe_mxfp4_layer_noalloc")
    return b


# ---- MXFP4 activations, and verification from probabilities ----------------

_Tensor = torch.Tensor
_functions = {}


def _enqueue(name, device, *args):
    """Call the library on `device`'s current stream (whatever device is current)."""
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    i = device.index
    if i == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(device):
            st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    if st:
        check(st, name)


def _want(t, name, dtype, shape, device):
    """_need, quickly where it holds: a call makes five of these checks and
    lasts a few microseconds itself."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and
            t.get_device() == device.index and t.is_contiguous()):
        _need(t, name, dtype, shape, device)


def _result(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, dtype, shape, device)
    return t


def _need_mx(codes, scales, name, shape, device):
    """codes uint8 [*shape[:-1], K/2] and scales uint8 [*shape[:-1], K/32] of an MXFP4 tensor."""
    rows, K = shape[:-1], shape[-1]
    _want(codes, name + "_codes", torch.uint8, rows + (K // 2,), device)
    _want(scales, name + "_scales", torch.uint8, rows + (K // 32,), device)


def _rank(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError("%s must be a tensor of %d dimensions" % (name, n))
    return t.shape


def mxfp4_gemm(a_codes, a_scales, b_codes, b_scales, dtype=torch.float32, out=None):
    """MXFP4 a [M, K] and b [N, K] (codes [rows, K/2], scales [rows, K/32]) ->
    a b^T [M, N] float32 or bfloat16."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dtype must be float32 or bfloat16")
    M, half = _rank(a_codes, "a_codes", 2)
    N, _ = _rank(b_codes, "b_codes", 2)
    K, dev = 2 * half, a_codes.device
    _need_mx(a_codes, a_scales, "a", (M, K), dev)
    _need_mx(b_codes, b_scales, "b", (N, K), dev)
    out = _result(out, "out", dtype, (M, N), dev)
    _enqueue("mxfp4_gemm", dev, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
             b_scales.data_ptr(), M, N, K, out.data_ptr(), BF16 if dtype == torch.bfloat16 else F32)
    return out


def _a4_gate_up_shapes(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes, w13_scales):
    T, half = _rank(x_codes, "x_codes", 2)
    E, two_i, _ = _rank(w13_codes, "w13_codes", 3)
    H, I, dev = 2 * half, two_i // 2, x_codes.device
    _need_mx(x_codes, x_scales, "x", (T, H), dev)
    _need_mx(w13_codes, w13_scales, "w13", (E, 2 * I, H), dev)
    _want(sorted_pairs, "sorted_pairs", torch.int32, (T * k,), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    return T, H, I, E, dev


def moe_mxfp4_a4_gate_up_swiglu(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes, w13_scales,
                                h=None):
    """MXFP4 x [T, H] -> h [T*k, I] bfloat16 (rows in sorted order)."""
    T, H, I, E, dev = _a4_gate_up_shapes(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes,
                                         w13_scales)
    h = _result(h, "h", torch.bfloat16, (T * k, I), dev)
    _enqueue("moe_mxfp4_a4_gate_up_swiglu", dev, x_codes.data_ptr(), x_scales.data_ptr(),
             sorted_pairs.data_ptr(), offsets.data_ptr(), T, H, I, E, k, w13_codes.data_ptr(),
             w13_scales.data_ptr(), h.data_ptr(), None, None)
    return h


def moe_mxfp4_a4_gate_up_swiglu_pack(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes,
                                     w13_scales, h_codes=None, h_scales=None):
    """moe_mxfp4_a4_gate_up_swiglu writing h in MXFP4 (mxfp4_pack of the
    bfloat16 h; where the sums are rounded in fp32 this call may round them in
    another order than that one) -> (h_codes [T*k, I/2], h_scales [T*k, I/32])."""
    T, H, I, E, dev = _a4_gate_up_shapes(x_codes, x_scales, sorted_pairs, offsets, k, w13_codes,
                                         w13_scales)
    h_codes = _result(h_codes, "h_codes", torch.uint8, (T * k, I // 2), dev)
    h_scales = _result(h_scales, "h_scales", torch.uint8, (T * k, I // 32), dev)
    _enqueue("moe_mxfp4_a4_gate_up_swiglu", dev, x_codes.data_ptr(), x_scales.data_ptr(),
             sorted_pairs.data_ptr(), offsets.data_ptr(), T, H, I, E, k, w13_codes.data_ptr(),
             w13_scales.data_ptr(), None, h_codes.data_ptr(), h_scales.data_ptr())
    return h_codes, h_scales


def moe_mxfp4_a4_down(h_codes, h_scales, offsets, k, w2_codes, w2_scales, y=None):
    """MXFP4 h [T*k, I] -> y [T*k, H] float32 (rows in sorted order)."""
    R, half = _rank(h_codes, "h_codes", 2)
    E, H, _ = _rank(w2_codes, "w2_codes", 3)
    I, dev = 2 * half, h_codes.device
    if k < 1 or R % k:
        raise ValueError("h must have T*k rows")
    _need_mx(h_codes, h_scales, "h", (R, I), dev)
    _need_mx(w2_codes, w2_scales, "w2", (E, H, I), dev)
    _want(offsets, "offsets", torch.int32, (E + 1,), dev)
    y = _result(y, "y", torch.float32, (R, H), dev)
    _enqueue("moe_mxfp4_a4_down", dev, h_codes.data_ptr(), h_scales.data_ptr(), offsets.data_ptr(),
             R // k, H, I, E, k, w2_codes.data_ptr(), w2_scales.data_ptr(), y.data_ptr())
    return y


class A4LayerBuffers:
    """Preallocated intermediates of one moe_mxfp4_a4_layer call."""

    def __init__(self, T, H, I, E, k, device):
        R = T * k
        z = dict(device=device)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, **z)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, **z)
        self.counts = torch.empty((E,), dtype=torch.int32, **z)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, **z)
        self.sorted_pairs = torch.empty((R,), dtype=torch.int32, **z)
        self.pair_to_row = torch.empty((R,), dtype=torch.int32, **z)
        self.x_codes = torch.empty((T, H // 2), dtype=torch.uint8, **z)
        self.x_scales = torch.empty((T, H // 32), dtype=torch.uint8, **z)
        self.h_codes = torch.empty((R, I // 2), dtype=torch.uint8, **z)
        self.h_scales = torch.empty((R, I // 32), dtype=torch.uint8, **z)
        self.y = torch.empty((R, H), dtype=torch.float32, **z)
        self.out = torch.empty((T, H), dtype=torch.float32, **z)
        nws = moe_permute_workspace_bytes(T, E, k)
        self.workspace = torch.empty(max(nws, 1), dtype=torch.uint8, **z)


def moe_mxfp4_a4_layer(x, logits, k, w13_codes, w13_scales, w2_codes, w2_scales, buffers=None):
    """The whole layer with MXFP4 activations in one C call (route, permute,
    pack x, gate/up with h in MXFP4, down, combine).

    Returns the A4LayerBuffers holding every intermediate; `.out` is the result."""
    T, H = _rank(x, "x", 2)
    E, two_i, _ = _rank(w13_codes, "w13_codes", 3)
    I, dev = two_i // 2, x.device
    _want(x, "x", torch.bfloat16, (T, H), dev)
    _want(logits, "logits", torch.float32, (T, E), dev)
    _need_mx(w13_codes, w13_scales, "w13", (E, 2 * I, H), dev)
    _need_mx(w2_codes, w2_scales, "w2", (E, H, I), dev)
    b = buffers if buffers is not None else A4LayerBuffers(T, H, I, E, k, dev)
    if (b.T, b.H, b.I, b.E, b.k) != (T, H, I, E, k) or b.out.device != dev:
        raise ValueError("buffers were made for another shape or device")
    _enqueue("moe_mxfp4_a4_layer", dev, _ptr(x), _ptr(logits), T, H, I, E, k, _ptr(w13_codes),
             _ptr(w13_scales), _ptr(w2_codes), _ptr(w2_scales), _ptr(b.topk_ids), _ptr(b.topk_w),
             _ptr(b.counts), _ptr(b.offsets), _ptr(b.sorted_pairs), _ptr(b.pair_to_row),
             _ptr(b.x_codes), _ptr(b.x_scales), _ptr(b.h_codes), _ptr(b.h_scales), _ptr(b.y),
             _ptr(b.out), _ptr(b.workspace), b.workspace.numel())
    return b


def dflash_verify_probs_workspace_bytes(B, L, V):
    return int(lib().dflash_verify_probs_workspace_bytes(B, L, V))


def dflash_verify_probs(target_probs, draft_probs, draft_tokens, uniforms, draft_len=None,
                        accept_len=None, next_token=None, workspace=None):
    """target_probs [B, L+1, V], draft_probs [B, L, V] (both float32 or both
    bfloat16), draft_tokens [B, L] int32, uniforms [B, L+1] f32, draft_len [B]
    int32 or None (every block has L tokens) -> (accept_len int32 [B],
    next_token int32 [B], -1 where no token has probability)."""
    B, L, V = _rank(draft_probs, "draft_probs", 3)
    dev, dtype = draft_probs.device, draft_probs.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("draft_probs must be float32 or bfloat16")
    _want(draft_probs, "draft_probs", dtype, (B, L, V), dev)
    _want(target_probs, "target_probs", dtype, (B, L + 1, V), dev)
    _want(draft_tokens, "draft_tokens", torch.int32, (B, L), dev)
    _want(uniforms, "uniforms", torch.float32, (B, L + 1), dev)
    if draft_len is not None:
        _want(draft_len, "draft_len", torch.int32, (B,), dev)
    accept_len = _result(accept_len, "accept_len", torch.int32, (B,), dev)
    next_token = _result(next_token, "next_token", torch.int32, (B,), dev)
    if workspace is None:
        need = dflash_verify_probs_workspace_bytes(B, L, V)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _need(workspace, "workspace", torch.uint8, None, dev)
    _enqueue("dflash_verify_probs", dev, target_probs.data_ptr(), draft_probs.data_ptr(),
             BF16 if dtype == torch.bfloat16 else F32, draft_tokens.data_ptr(), _ptr(draft_len),
             uniforms.data_ptr(), B, L, V, accept_len.data_ptr(), next_token.data_ptr(), _ptr(workspace),
             0 if workspace is None else workspace.numel())
    return accept_len, next_token


def mxm_stream_xor(src, result, nontemporal=False):
    """Streaming-read probe (a measurement aid): XOR every 32-bit word of the
    contiguous tensor `src` (byte size a multiple of 16) into `result`, an
    int32 tensor of one element that the caller initialises."""
    if not isinstance(src, torch.Tensor) or src.device.type != "cuda" or not src.is_contiguous():
        raise ValueError("src must be a contiguous GPU tensor")
    _need(result, "result", torch.int32, (1,), src.device)
    nbytes = src.numel() * src.element_size()
    check(lib().mxm_stream_xor(_ptr(src), nbytes, 1 if nontemporal else 0, _ptr(result),
                               _stream()), "mxm_stream_xor")
    return result

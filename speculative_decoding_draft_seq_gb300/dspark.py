"""Python binding of the DSpark C-ABI library (libdspark.so).

Argument marshalling only: every step of the round runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (device memory and streams are
PyTorch's); the binding passes their data pointers and the current stream's
handle to the C entry points declared in include/dspark.h. If the library is
missing the import fails: there is no fallback implementation.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark.so")

OK, ERR_INVALID_ARG, ERR_NONFINITE, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_RANGE, ERR_TOO_LARGE, \
    ERR_CAPACITY = range(9)
FP32, BF16 = 0, 1
CAUSAL, LAGGED, ALL = 0, 1, 2


class DSparkError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    i32, u64, f32, vp, sz = ctypes.c_int32, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    lib.dspark_workspace_bytes.restype = sz
    lib.dspark_workspace_bytes.argtypes = [i32] * 6
    lib.dspark_workspace_init.restype = i32
    lib.dspark_workspace_init.argtypes = [vp, sz, vp]
    lib.dspark_draft_sequential.restype = i32
    lib.dspark_draft_sequential.argtypes = [i32] * 5 + [vp] * 4 + [f32, u64] + [vp] * 3 + [vp, sz, vp]
    lib.dspark_schedule.restype = i32
    lib.dspark_schedule.argtypes = [i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.dspark_schedule_static.restype = i32
    lib.dspark_schedule_static.argtypes = [i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.dspark_verify.restype = i32
    lib.dspark_verify.argtypes = [i32] * 5 + [vp] * 9 + [f32, u64] + [vp] * 3 + [vp, sz, vp]
    lib.dspark_round.restype = i32
    lib.dspark_round.argtypes = ([i32] * 5 + [vp] * 5 + [vp, vp, vp, i32, i32, f32, u64] +
                                 [vp] * 9 + [vp, sz, vp])
    lib.dspark_draft_sequential_gated.restype = i32
    lib.dspark_draft_sequential_gated.argtypes = [i32] * 5 + [vp] * 5 + [f32, u64] + [vp] * 3 + [vp, sz, vp]
    lib.dspark_verify_gated.restype = i32
    lib.dspark_verify_gated.argtypes = [i32] * 5 + [vp] * 10 + [f32, u64] + [vp] * 3 + [vp, sz, vp]
    lib.dspark_round_gated.restype = i32
    lib.dspark_round_gated.argtypes = ([i32] * 5 + [vp] * 6 + [vp, vp, vp, i32, i32, f32, u64] +
                                       [vp] * 9 + [vp, sz, vp])
    lib.dspark_lm_head.restype = i32
    lib.dspark_lm_head.argtypes = [i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.dspark_copy_scheduled_rows.restype = i32
    lib.dspark_copy_scheduled_rows.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
    lib.dspark_wait_selftest.restype = i32
    lib.dspark_wait_selftest.argtypes = [i32, vp, sz, vp]
    lib.dspark_acceptance_labels.restype = i32
    lib.dspark_acceptance_labels.argtypes = [i32] * 5 + [vp] * 7 + [f32, vp, vp, sz, vp]
    lib.dspark_sts_scratch_bytes.restype = sz
    lib.dspark_sts_scratch_bytes.argtypes = [i32] * 4
    lib.dspark_sts_fit.restype = i32
    lib.dspark_sts_fit.argtypes = [i32, i32, vp, vp, i32, vp, i32, vp, vp, vp, sz, vp]
    lib.dspark_sts_status.restype = i32
    lib.dspark_sts_status.argtypes = [vp, vp]
    lib.dspark_sts_apply.restype = i32
    lib.dspark_sts_apply.argtypes = [i32, i32, vp, vp, vp, vp]
    i64 = ctypes.c_int64
    lib.dspark_page_plan.restype = i32
    lib.dspark_page_plan.argtypes = [i32] * 5 + [vp] * 9 + [vp, sz, vp]
    lib.dspark_kv_append.restype = i32
    lib.dspark_kv_append.argtypes = [i32] * 4 + [vp] * 3 + [i64] + [vp] * 2 + [vp, sz, vp]
    lib.dspark_attention_workspace_bytes.restype = sz
    lib.dspark_attention_workspace_bytes.argtypes = [i32] * 5
    lib.dspark_prefix_attention.restype = i32
    lib.dspark_prefix_attention.argtypes = [i32] * 9 + [vp] * 7 + [f32] + [vp] * 2 + [vp, sz, vp]
    lib.dspark_sample.restype = i32
    lib.dspark_sample.argtypes = [i32] * 3 + [vp] * 8 + [vp, sz, vp]
    lib.dspark_truncate.restype = i32
    lib.dspark_truncate.argtypes = [i32] * 3 + [vp] * 6 + [vp, sz, vp]
    lib.dspark_device_status.restype = i32
    lib.dspark_device_status.argtypes = [vp, vp]
    lib.dspark_status_string.restype = ctypes.c_char_p
    lib.dspark_status_string.argtypes = [i32]
    lib.dspark_last_launch_count.restype = i32
    lib.dspark_last_launch_count.argtypes = []
    return lib


lib = _load()


def status_string(status):
    return lib.dspark_status_string(int(status)).decode()


def last_launch_count():
    return int(lib.dspark_last_launch_count())


_I32, _F32, _F64, _U8 = torch.int32, torch.float32, torch.float64, torch.uint8
_I64, _BF16 = torch.int64, torch.bfloat16


def _ptr(t, dtype=None, host=False):
    """Data pointer of a dense tensor for the C ABI, which takes row-major arrays without strides:
    a non-contiguous view, a tensor on the wrong side of the host/device split or (where the entry
    point fixes it) the wrong element type is refused here rather than read or written wrongly."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the C ABI takes dense row-major arrays)")
    if t.is_cuda == host:
        raise ValueError("expected a host tensor" if host else "expected a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"logits/weights must be bfloat16 or float32, got {t.dtype}")


def _check(status, where):
    if status != OK:
        raise DSparkError(status, where)


def workspace_bytes(R, gamma, V, rank, dtype, n_table):
    return int(lib.dspark_workspace_bytes(R, gamma, V, rank, dtype, n_table))


def _aligned_workspace(n, device, stream):
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    _check(lib.dspark_workspace_init(_ptr(ws, _U8), n, _stream(stream)), "dspark_workspace_init")
    return ws


def new_workspace(R, gamma, V, rank, dtype, n_table, device="cuda", stream=None):
    """Allocates (with PyTorch) and clears a workspace for these sizes."""
    n = workspace_bytes(R, gamma, V, rank, dtype, n_table)
    return _aligned_workspace(n, device, stream)


def draft_sequential(base, anchor, W1, W2, temperature, seed, tokens, q_tok, q_stats, ws, stream=None):
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_draft_sequential(R, gamma, V, rank, _dtype_code(base), _ptr(base), _ptr(anchor, _I32),
                                       _ptr(W1), _ptr(W2), float(temperature), int(seed), _ptr(tokens, _I32),
                                       _ptr(q_tok, _F32), _ptr(q_stats, _F32), _ptr(ws, _U8), ws.numel(),
                                       _stream(stream)), "dspark_draft_sequential")


def draft_sequential_gated(base, anchor, W1, gate, W2, temperature, seed, tokens, q_tok, q_stats, ws,
                           stream=None):
    """Drafting with the recurrent (gated) head; `gate` [V, rank] like W1."""
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_draft_sequential_gated(R, gamma, V, rank, _dtype_code(base), _ptr(base), _ptr(anchor, _I32),
                                             _ptr(W1), _ptr(gate), _ptr(W2), float(temperature), int(seed),
                                             _ptr(tokens, _I32), _ptr(q_tok, _F32), _ptr(q_stats, _F32),
                                             _ptr(ws, _U8), ws.numel(), _stream(stream)),
           "dspark_draft_sequential_gated")


def lm_head(hidden, lm_head_w, logits, ws, stream=None):
    """Base logits bf16(hidden . lm_head): hidden [..., d], lm_head [d, V],
    logits [..., V] (bf16 tensors; the leading dimensions are flattened)."""
    d, V = lm_head_w.shape
    M = hidden.numel() // d
    _check(lib.dspark_lm_head(M, d, V, _ptr(hidden), _ptr(lm_head_w), _ptr(logits), _ptr(ws, _U8), ws.numel(),
                              _stream(stream)), "dspark_lm_head")


def schedule(conf, conf_lagged, sps, mode, sched_len, K, tau_theta, ws, stream=None):
    R, gamma = conf.shape
    _check(lib.dspark_schedule(R, gamma, _ptr(conf, _F32), _ptr(conf_lagged, _F32), _ptr(sps, _F32), sps.numel(),
                               int(mode), _ptr(sched_len, _I32), _ptr(K, _I32), _ptr(tau_theta, _F64),
                               _ptr(ws, _U8), ws.numel(), _stream(stream)), "dspark_schedule")


def schedule_static(conf, conf_lagged, sps, mode, sched_len, K, tau_theta, device_status=None,
                    stream=None):
    """dspark_schedule_static: the scheduler without a workspace (fixed library
    scratch, R * gamma <= 16384). Returns the C status code without raising."""
    R, gamma = conf.shape
    return int(lib.dspark_schedule_static(R, gamma, _ptr(conf, _F32), _ptr(conf_lagged, _F32), _ptr(sps, _F32),
                                          sps.numel(), int(mode), _ptr(sched_len, _I32), _ptr(K, _I32),
                                          _ptr(tau_theta, _F64), _ptr(device_status), _stream(stream)))


def verify(target, base, anchor, W1, W2, tokens, q_tok, q_stats, sched_len, temperature, seed,
           out_tokens, accepted_len, p_tok, ws, stream=None):
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_verify(R, gamma, V, rank, _dtype_code(base), _ptr(target), _ptr(base), _ptr(anchor, _I32),
                             _ptr(W1), _ptr(W2), _ptr(tokens, _I32), _ptr(q_tok, _F32), _ptr(q_stats, _F32),
                             _ptr(sched_len, _I32), float(temperature), int(seed), _ptr(out_tokens, _I32),
                             _ptr(accepted_len, _I32), _ptr(p_tok, _F32), _ptr(ws, _U8), ws.numel(),
                             _stream(stream)), "dspark_verify")


def verify_gated(target, base, anchor, W1, gate, W2, tokens, q_tok, q_stats, sched_len, temperature, seed,
                 out_tokens, accepted_len, p_tok, ws, stream=None):
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_verify_gated(R, gamma, V, rank, _dtype_code(base), _ptr(target), _ptr(base),
                                   _ptr(anchor, _I32), _ptr(W1), _ptr(gate), _ptr(W2), _ptr(tokens, _I32),
                                   _ptr(q_tok, _F32), _ptr(q_stats, _F32), _ptr(sched_len, _I32),
                                   float(temperature), int(seed), _ptr(out_tokens, _I32), _ptr(accepted_len, _I32),
                                   _ptr(p_tok, _F32), _ptr(ws, _U8), ws.numel(), _stream(stream)),
           "dspark_verify_gated")


def acceptance_labels(target, base, anchor, W1, W2, tokens, q_stats, temperature, labels, ws, stream=None):
    """dspark_acceptance_labels: labels [R, gamma] float32 = 1 - TV(P_{k-1}, Q_k) per position."""
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_acceptance_labels(R, gamma, V, rank, _dtype_code(base), _ptr(target), _ptr(base),
                                        _ptr(anchor, _I32), _ptr(W1), _ptr(W2), _ptr(tokens, _I32),
                                        _ptr(q_stats, _F32), float(temperature), _ptr(labels, _F32), _ptr(ws, _U8),
                                        ws.numel(), _stream(stream)), "dspark_acceptance_labels")


def sts_fit(conf, accepted, grid, n_bins, temperature, ece=None, stream=None):
    """dspark_sts_fit with a scratch it allocates (PyTorch); returns the device status."""
    N, gamma = conf.shape
    n = int(lib.dspark_sts_scratch_bytes(N, gamma, grid.numel(), n_bins))
    if n == 0:
        raise DSparkError(ERR_INVALID_ARG, "dspark_sts_scratch_bytes")
    raw = torch.empty(n + 256, dtype=torch.uint8, device=conf.device)
    off = (-raw.data_ptr()) % 256
    scratch = raw[off:off + n]
    _check(lib.dspark_sts_fit(N, gamma, _ptr(conf, _F32), _ptr(accepted, _I32), grid.numel(), _ptr(grid, _F32),
                              n_bins, _ptr(temperature, _F32), _ptr(ece, _F32), _ptr(scratch, _U8), n,
                              _stream(stream)), "dspark_sts_fit")
    return int(lib.dspark_sts_status(_ptr(scratch, _U8), _stream(stream)))


def sts_apply(conf, temperature, conf_out, stream=None):
    R, gamma = conf.shape
    _check(lib.dspark_sts_apply(R, gamma, _ptr(conf, _F32), _ptr(temperature, _F32), _ptr(conf_out, _F32),
                                _stream(stream)), "dspark_sts_apply")


def round_(base, target, anchor, W1, W2, conf, conf_lagged, sps, mode, temperature, seed, out, ws,
           stream=None):
    """One whole round; `out` is a RoundOutputs holding the output tensors."""
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_round(R, gamma, V, rank, _dtype_code(base), _ptr(base), _ptr(target), _ptr(anchor, _I32),
                            _ptr(W1), _ptr(W2), _ptr(conf, _F32), _ptr(conf_lagged, _F32), _ptr(sps, _F32),
                            sps.numel(), int(mode), float(temperature), int(seed), _ptr(out.tokens, _I32),
                            _ptr(out.q_tok, _F32), _ptr(out.q_stats, _F32), _ptr(out.sched_len, _I32),
                            _ptr(out.K, _I32), _ptr(out.tau_theta, _F64), _ptr(out.out_tokens, _I32),
                            _ptr(out.accepted_len, _I32), _ptr(out.p_tok, _F32), _ptr(ws, _U8), ws.numel(),
                            _stream(stream)), "dspark_round")


def round_gated(base, target, anchor, W1, gate, W2, conf, conf_lagged, sps, mode, temperature, seed, out, ws,
                stream=None):
    """One whole round with the recurrent (gated) head."""
    R, gamma, V = base.shape
    rank = W1.shape[1]
    _check(lib.dspark_round_gated(R, gamma, V, rank, _dtype_code(base), _ptr(base), _ptr(target),
                                  _ptr(anchor, _I32), _ptr(W1), _ptr(gate), _ptr(W2), _ptr(conf, _F32),
                                  _ptr(conf_lagged, _F32), _ptr(sps, _F32), sps.numel(), int(mode),
                                  float(temperature), int(seed), _ptr(out.tokens, _I32), _ptr(out.q_tok, _F32),
                                  _ptr(out.q_stats, _F32), _ptr(out.sched_len, _I32), _ptr(out.K, _I32),
                                  _ptr(out.tau_theta, _F64), _ptr(out.out_tokens, _I32),
                                  _ptr(out.accepted_len, _I32), _ptr(out.p_tok, _F32), _ptr(ws, _U8), ws.numel(),
                                  _stream(stream)), "dspark_round_gated")


def copy_scheduled_rows(host_target, device_target, host_sched_len, stream=None):
    """Host-to-device copy of target rows 0..L_r of every request (host_target pinned)."""
    R, g1, V = host_target.shape
    _check(lib.dspark_copy_scheduled_rows(R, g1 - 1, V, _dtype_code(host_target),
                                          _ptr(host_target, host=True), _ptr(device_target),
                                          _ptr(host_sched_len, _I32, host=True), _stream(stream)),
           "dspark_copy_scheduled_rows")


# Calls of a serving step are short: these helpers do what _ptr and _stream do with fewer Python steps.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _addr(t, dtype):
    """Device address of a dense CUDA tensor of this type; refuses what _ptr refuses."""
    if t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, dtype).value


def _shapes(**named):
    """Refuses tensors whose shape is not the one given: name=(tensor, shape), None for any size."""
    for name, (t, want) in named.items():
        if len(t.shape) != len(want) or any(w is not None and w != n for n, w in zip(t.shape, want)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                             f"{tuple('any' if w is None else w for w in want)}")


def page_plan(cached_len, new_len, free_pages, page_size, block_table, q_start, kv_len, positions, slots, used, ws,
              stream=None):
    """Cache pages and slots of new_len[r] tokens a request: fills the new entries of block_table
    [R, max_pages] from free_pages, and q_start [R+1], kv_len [R], positions and slots [capacity]
    (int32, int64) and used [1]. Tokens past the capacity are left out of all of them (ERR_CAPACITY)."""
    R, max_pages = block_table.shape
    capacity = positions.numel()
    if (cached_len.shape != (R,) or new_len.shape != (R,) or q_start.shape != (R + 1,) or kv_len.shape != (R,) or
            slots.shape != (capacity,) or used.numel() < 1):
        _shapes(cached_len=(cached_len, (R,)), new_len=(new_len, (R,)), q_start=(q_start, (R + 1,)),
                kv_len=(kv_len, (R,)), slots=(slots, (capacity,)), used=(used, (1,)))
    status = lib.dspark_page_plan(R, page_size, max_pages, free_pages.numel(), capacity, _addr(cached_len, _I32),
                                  _addr(new_len, _I32), _addr(free_pages, _I32), _addr(block_table, _I32),
                                  _addr(q_start, _I32), _addr(kv_len, _I32), _addr(positions, _I32),
                                  _addr(slots, _I64), _addr(used, _I32), _addr(ws, _U8), ws.numel(),
                                  _raw_stream(stream))
    if status:
        _check(status, "dspark_page_plan")


def kv_append(k, v, slots, k_cache, v_cache, ws, stream=None):
    """k_cache[slots[t]] = k[t] and the same for v: k, v [T, Hkv, D], caches
    [pages, page_size, Hkv, D] (any leading dimensions), slots [T] int64; negative slots are skipped."""
    T, Hkv, D = k.shape
    if v.shape != (T, Hkv, D) or slots.shape != (T,):
        _shapes(v=(v, (T, Hkv, D)), slots=(slots, (T,)))
    if k_cache.shape != v_cache.shape or k_cache.shape[-2:] != (Hkv, D):
        raise ValueError("k_cache and v_cache must have one shape that ends in (Hkv, D)")
    dt = k.dtype
    status = lib.dspark_kv_append(T, Hkv, D, _dtype_code(k), _addr(k, dt), _addr(v, dt), _addr(slots, _I64),
                                  k_cache.numel() // (Hkv * D), _addr(k_cache, dt), _addr(v_cache, dt),
                                  _addr(ws, _U8), ws.numel(), _raw_stream(stream))
    if status:
        _check(status, "dspark_kv_append")


def attention_workspace_bytes(R, T, Hq, Hkv, D):
    return int(lib.dspark_attention_workspace_bytes(R, T, Hq, Hkv, D))


def new_attention_workspace(R, T, Hq, Hkv, D, device="cuda", stream=None):
    """Allocates (with PyTorch) and clears a workspace for prefix_attention calls of up to R
    requests and T query tokens."""
    n = attention_workspace_bytes(R, T, Hq, Hkv, D)
    if n == 0:
        raise DSparkError(ERR_INVALID_ARG, "dspark_attention_workspace_bytes")
    return _aligned_workspace(n, device, stream)


def prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, q_start, kv_len, scale, out, ws,
                     lse=None, stream=None):
    """Attention of q [T, Hq, D] over the shared prefix and each request's own pages (caches
    [n_pages, page_size, Hkv, D], block_table [R, max_pages]); writes out like q and, unless None,
    lse [T, Hq] float32."""
    T, Hq, D = q.shape
    n_pages, page, Hkv, Dk = k_cache.shape
    R, max_pages = block_table.shape
    if (Dk != D or v_cache.shape != k_cache.shape or out.shape != q.shape or q_start.shape != (R + 1,) or
            kv_len.shape != (R,) or (lse is not None and lse.shape != (T, Hq))):
        _shapes(k_cache=(k_cache, (None, None, None, D)), v_cache=(v_cache, tuple(k_cache.shape)),
                out=(out, (T, Hq, D)), q_start=(q_start, (R + 1,)), kv_len=(kv_len, (R,)),
                **({} if lse is None else {"lse": (lse, (T, Hq))}))
    if prefix_len > 0 and prefix_pages.numel() * page < prefix_len:
        raise ValueError("prefix_pages does not cover prefix_len")
    status = lib.dspark_prefix_attention(R, T, Hq, Hkv, D, page, n_pages, max_pages, prefix_len, _addr(q, _BF16),
                                         _addr(k_cache, _BF16), _addr(v_cache, _BF16),
                                         _addr(prefix_pages, _I32) if prefix_len > 0 else None,
                                         _addr(block_table, _I32), _addr(q_start, _I32), _addr(kv_len, _I32), scale,
                                         _addr(out, _BF16), None if lse is None else _addr(lse, _F32), _addr(ws, _U8),
                                         ws.numel(), _raw_stream(stream))
    if status:
        _check(status, "dspark_prefix_attention")


def _rule(logits, temperature, top_k, top_p, min_p):
    N, V = logits.shape
    if temperature.shape != (N,) or top_k.shape != (N,) or top_p.shape != (N,) or min_p.shape != (N,):
        _shapes(temperature=(temperature, (N,)), top_k=(top_k, (N,)), top_p=(top_p, (N,)), min_p=(min_p, (N,)))
    return (N, V, _dtype_code(logits), _addr(logits, logits.dtype), _addr(temperature, _F32), _addr(top_k, _I32),
            _addr(top_p, _F32), _addr(min_p, _F32))


def sample(logits, temperature, top_k, top_p, min_p, u, tokens, ws, prob=None, stream=None):
    """One token a row of logits [N, V] by temperature, top-k, top-p and min-p (one of each a row)
    from the uniforms u [N] float64; tokens [N] int32, prob [N] float32 or None."""
    rule = _rule(logits, temperature, top_k, top_p, min_p)
    N = rule[0]
    if u.shape != (N,) or tokens.shape != (N,) or (prob is not None and prob.shape != (N,)):
        _shapes(u=(u, (N,)), tokens=(tokens, (N,)), **({} if prob is None else {"prob": (prob, (N,))}))
    status = lib.dspark_sample(*rule, _addr(u, _F64), _addr(tokens, _I32), None if prob is None else _addr(prob, _F32),
                               _addr(ws, _U8), ws.numel(), _raw_stream(stream))
    if status:
        _check(status, "dspark_sample")


def truncate(logits, temperature, top_k, top_p, min_p, out, ws, stream=None):
    """out [N, V]: logits with every entry outside the rule's kept set at the type's lowest value. The kept ones are not
    divided by the temperature: verify applies its own, one for all rows."""
    rule = _rule(logits, temperature, top_k, top_p, min_p)
    if out.shape != logits.shape:
        _shapes(out=(out, tuple(logits.shape)))
    status = lib.dspark_truncate(*rule, _addr(out, logits.dtype), _addr(ws, _U8), ws.numel(), _raw_stream(stream))
    if status:
        _check(status, "dspark_truncate")


def wait_selftest(which, ws, stream=None):
    """A bounded device wait (0: grid barrier, 1: mbarrier, 2: counter poll) on a condition nothing meets; it
    gives up and records ERR_TIMEOUT in the workspace's status word."""
    _check(lib.dspark_wait_selftest(int(which), _ptr(ws, _U8), ws.numel(), _stream(stream)), "dspark_wait_selftest")


def device_status(ws, stream=None):
    return int(lib.dspark_device_status(_ptr(ws, _U8), _stream(stream)))


class RoundOutputs:
    """Device output tensors of one round for R requests and block length gamma."""

    def __init__(self, R, gamma, device="cuda"):
        i32, f32 = torch.int32, torch.float32
        self.tokens = torch.zeros((R, gamma), dtype=i32, device=device)
        self.q_tok = torch.zeros((R, gamma), dtype=f32, device=device)
        self.q_stats = torch.zeros((R, gamma, 2), dtype=f32, device=device)
        self.sched_len = torch.zeros((R,), dtype=i32, device=device)
        self.K = torch.zeros((1,), dtype=i32, device=device)
        self.tau_theta = torch.zeros((2,), dtype=torch.float64, device=device)
        self.out_tokens = torch.zeros((R, gamma + 1), dtype=i32, device=device)
        self.accepted_len = torch.zeros((R,), dtype=i32, device=device)
        self.p_tok = torch.zeros((R, gamma), dtype=f32, device=device)

    def host(self):
        return {k: v.cpu().numpy() for k, v in vars(self).items()}
